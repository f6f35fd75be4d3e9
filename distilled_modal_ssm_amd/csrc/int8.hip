// int8.hip -- products in 8-bit integers: rows of activations and of weights as
// whole multiples of a scale of their own, their products summed exactly in 32 bits
// on the matrix cores, the scales applied to the sums.
#include <type_traits>
#include <utility>

#include "hm_internal.hpp"

namespace hm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(uint4 a, uint4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Rows are held in blocks of 16 rows by 64 columns, 1024 bytes each.  Place of the
// 16-byte chunk c of a block's row r: the LDS serves a 16-byte read of a wave 16 lanes at
// a time, from 0-3, 12-15, 20-23 and 24-27 on; with a fragment's rows l % 16 and chunks
// l / 16, those and all others that go together fall on all 64 banks.
__device__ __forceinline__ int place(int r, int c) {
    const int fours = (r >> 2) & 3;  // 0 1 2 3 -> 0 2 3 1
    return 64 * r + 16 * (c ^ (((fours << 1) ^ (3 * (fours >> 1))) & 3));
}

__device__ __forceinline__ int64_t block_of(int64_t row, int64_t K) { return (row >> 4) * ((K + 63) >> 6) * 1024; }

// ------------------------------------------------------------------ rows in 8 bits

// rint(127 x / amax), the integer of the exact quotient: in float32, off by less than
// 127 * 2^-22, and again in float64 where that could matter (its product is exact, and
// a quotient of two 24-bit numbers is never nearer to a border than 2^-32 without
// being on it).
__device__ __forceinline__ int quantized(float x, float amax, float inverse) {
    const float r = x * inverse, n = rintf(r);
    if (fabsf(r - n) < 0.4999f && amax > 1e-30f) return (int)n;
    return (int)rint((double)x * 127.0 / (double)amax);
}

struct RowStat {
    uint32_t top;  // bits of the largest magnitude; NaN and infinities come last
    float sum;     // of squares
};

__device__ __forceinline__ void take(RowStat &s, float x) {
    const uint32_t bits = __float_as_uint(x) & 0x7fffffffu;
    s.top = bits > s.top ? bits : s.top;
    s.sum = fmaf(x, x, s.sum);
}

// The statistics of W waves' row, joined in all of them.
template <int W> __device__ __forceinline__ RowStat joined(RowStat s) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        const uint32_t top = __shfl_xor(s.top, m);
        s.top = top > s.top ? top : s.top;
        s.sum += __shfl_xor(s.sum, m);
    }
    if constexpr (W > 1) {
        __shared__ RowStat all[W];
        if (threadIdx.x % kWave == 0) all[threadIdx.x / kWave] = s;
        __syncthreads();
        s = all[0];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            s.top = all[w].top > s.top ? all[w].top : s.top;
            s.sum += all[w].sum;
        }
    }
    return s;
}

// The row's scale; 0 of a row of zeros, without eps too.
__device__ __forceinline__ float row_scale(const QuantArgs &a, const RowStat &s) {
    float scale = __uint_as_float(s.top) / 127.0f;
    if (a.rms && s.top > 0) scale = scale / sqrtf(s.sum / (float)a.K + a.eps);
    return s.top < 0x7f800000u ? scale : __builtin_nanf("");
}

// Whether the row's squares have to be summed again, in float64, and its scale formed
// there: where float32's sum has left its range; where amax / 127 is subnormal, and loses
// digits that the root gives back; where squares below 2^-149 could count, of rows below
// 2^-50 (K of them are less than 2^-132, and the largest square is 2^-100 at least)
// without an eps that is larger than any of them.  (Behind everything else, as one branch
// of the wave: with the two scales side by side, 5 x 6144 x 2048 took 0.4 us of 8.7 more.)
__device__ __forceinline__ bool sum_again(const QuantArgs &a, const RowStat &s) {
    if (!a.rms) return false;
    const uint32_t low = __float_as_uint(a.eps < 0x1p-100f ? 0x1p-50f : 0x1p-118f);
    return __builtin_amdgcn_readfirstlane((int)(s.top - 1 < low - 1 || !(s.sum < __builtin_inff())));
}

// That scale, by W waves, in all of them.  The row is read again, a value at a time: kept
// in registers it would take them from every row.
template <int ACT, int W>
__device__ __forceinline__ float row_scale_again(const QuantArgs &a, int64_t m, uint32_t top) {
    const typename Act<ACT>::T *x = static_cast<const typename Act<ACT>::T *>(a.x) + m * a.ldx;
    double sum = 0.0;
#pragma nounroll
    for (int64_t k = threadIdx.x % (W * kWave); k < a.K; k += W * kWave) {
        const double v = Act<ACT>::ld(x + k);
        sum = fma(v, v, sum);
    }
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
    if constexpr (W > 1) {
        __shared__ double all[W];
        if (threadIdx.x % kWave == 0) all[threadIdx.x / kWave] = sum;
        __syncthreads();
        sum = all[0];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += all[w];
    }
    if (top >= 0x7f800000u) return __builtin_nanf("");
    return (float)(__uint_as_float(top) / 127.0 / sqrt(sum / (double)a.K + (double)a.eps));
}

// E values' integers as bytes.
template <int E> __device__ __forceinline__ void quantize(const float (&x)[E], float amax, float inverse, int (&n)[E]) {
    bool sure = amax > 1e-30f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float r = x[e] * inverse, near = rintf(r);
        n[e] = (int)near;
        sure = sure && fabsf(r - near) < 0.4999f;
    }
    if (!sure) {
#pragma unroll
        for (int e = 0; e < E; ++e) n[e] = quantized(x[e], amax, inverse);
    }
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A row's 16 bytes `at`, `at` + lanes, .. as they lie, at any alignment; what is past the
// row's end reads as 0.  (Bounds count 4 bytes: the last of an odd number of bfloat16
// values comes by itself.)  One value at a time, where rows are not aligned, a call of
// 9627 x 112 x 5517 bfloat16 took 134 us, so 63.
template <int ACT, int N>
__device__ __forceinline__ void load_row(const void *row, int K, int at, int lanes, u32x4 (&piece)[N]) {
    const auto x = make_region(row, (uint32_t)K * Act<ACT>::kBytes & ~3u);
#pragma unroll
    for (int k = 0; k < N; ++k) piece[k] = __builtin_amdgcn_raw_buffer_load_b128(x, 16 * (k * lanes + at), 0, 0);
    if constexpr (ACT == kBF16) {
        if (K % 2 == 0) return;
        const uint32_t last = static_cast<const uint16_t *>(row)[K - 1];
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (8 * (k * lanes + at) + 2 * e == K - 1) piece[k][e] = last;
    }
}

template <int ACT, int N> __device__ __forceinline__ void piece_values(const u32x4 (&piece)[N], int k, float *v) {
#pragma unroll
    for (int e = 0; e < 16 / Act<ACT>::kBytes; ++e) {
        if constexpr (ACT == kBF16) v[e] = e % 2 ? bf16_hi(piece[k][e / 2]) : bf16_lo(piece[k][e / 2]);
        else v[e] = __uint_as_float(piece[k][e]);
    }
}

template <int ACT, int N> __device__ __forceinline__ void take_row(RowStat &s, const u32x4 (&piece)[N]) {
    constexpr int E = 16 / Act<ACT>::kBytes;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float v[E];
        piece_values<ACT>(piece, k, v);
#pragma unroll
        for (int e = 0; e < E; ++e) take(s, v[e]);
    }
}

// The integers of load_row's values, to row r of blocks that have `end` columns.
template <int ACT, int N>
__device__ __forceinline__ void put_row(int8_t *blocks, int r, int end, int at, int lanes, const u32x4 (&piece)[N], const RowStat &s) {
    constexpr int E = 16 / Act<ACT>::kBytes;
    const bool some = s.top > 0 && s.top < 0x7f800000u;
    const float amax = __uint_as_float(s.top), inverse = 127.0f / amax;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int col = E * (k * lanes + at);
        if (col >= end) break;
        uint32_t out[E / 4] = {};
        if (some) {
            float v[E];
            int n[E];
            piece_values<ACT>(piece, k, v);
            quantize(v, amax, inverse, n);
#pragma unroll
            for (int e = 0; e < E; ++e) out[e / 4] |= (uint32_t)(n[e] & 255) << (8 * (e % 4));
        }
        int8_t *q = blocks + col / 64 * 1024 + place(r, col % 64 / 16) + col % 16;
        if constexpr (E == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(out[0], out[1]);
        else *reinterpret_cast<uint32_t *>(q) = out[0];
    }
}

// A row in the registers of W waves, N pieces of 16 bytes a lane, read once.
template <int ACT, int N, int W>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
    constexpr int kLanes = W * kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t m = W > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
    if (m >= a.M) return;
    const int lane = W > 1 ? (int)threadIdx.x : (int)threadIdx.x % kWave, K = (int)a.K;
    u32x4 piece[N];
    load_row<ACT>(static_cast<const unsigned char *>(a.x) + m * a.ldx * Act<ACT>::kBytes, K, lane, kLanes, piece);
    RowStat s{0, 0.0f};
    take_row<ACT>(s, piece);
    s = joined<W>(s);
    put_row<ACT>(a.q + block_of(m, K), (int)(m % 16), (K + 63) / 64 * 64, lane, kLanes, piece, s);
    if (lane == 0) a.scale[m] = row_scale(a, s);
    if (__builtin_expect(sum_again(a, s), 0)) {
        const float scale = row_scale_again<ACT, W>(a, m, s.top);
        if (lane == 0) a.scale[m] = scale;
    }
}

// Longer rows: one workgroup a row, which is read twice, the second time from the caches
// (1804 x 24482 float32: 57 us less than one value at a time).
template <int ACT>
__global__ __launch_bounds__(256) void quantize_long_rows_kernel(QuantArgs a) {
    constexpr int EB = Act<ACT>::kBytes, N = 4, kTurn = N * 256 * 16 / EB;
    const int64_t m = blockIdx.x;
    const unsigned char *x = static_cast<const unsigned char *>(a.x) + m * a.ldx * EB;
    const int tid = threadIdx.x, K = (int)a.K, end = (K + 63) / 64 * 64;
    RowStat s{0, 0.0f};
    u32x4 piece[N];
    for (int k = 0; k < K; k += kTurn) {
        load_row<ACT>(x + (int64_t)k * EB, K - k < kTurn ? K - k : kTurn, tid, 256, piece);
        take_row<ACT>(s, piece);
    }
    s = joined<4>(s);
    int8_t *q = a.q + block_of(m, K);
    for (int k = 0; k < K; k += kTurn) {
        load_row<ACT>(x + (int64_t)k * EB, K - k < kTurn ? K - k : kTurn, tid, 256, piece);
        put_row<ACT>(q + (int64_t)k / 64 * 1024, (int)(m % 16), end - k, tid, 256, piece, s);
    }
    if (tid == 0) a.scale[m] = row_scale(a, s);
    if (__builtin_expect(sum_again(a, s), 0)) {
        const float scale = row_scale_again<ACT, 4>(a, m, s.top);
        if (tid == 0) a.scale[m] = scale;
    }
}

template <int ACT> void launch_quantize(const QuantArgs &a, hipStream_t stream) {
    constexpr int EB = Act<ACT>::kBytes, E = 16 / EB;
    const dim3 rows((unsigned)a.M);
    if (a.K > 16 * E * 256) return quantize_long_rows_kernel<ACT><<<rows, 256, 0, stream>>>(a);
    if (a.M >= 1024 && a.K <= 4 * E * kWave)
        return quantize_rows_kernel<ACT, 4, 1><<<dim3((unsigned)((a.M + 3) / 4)), 256, 0, stream>>>(a);
    if (a.K <= E * 256) return quantize_rows_kernel<ACT, 1, 4><<<rows, 256, 0, stream>>>(a);
    if (a.K <= 4 * E * 256) return quantize_rows_kernel<ACT, 4, 4><<<rows, 256, 0, stream>>>(a);
    quantize_rows_kernel<ACT, 16, 4><<<rows, 256, 0, stream>>>(a);
}

// ------------------------------------------------------------------ products, tiles

// step(B), step(B + 1), .. step(E - 1) until `left` of them are done; whether they are.
template <int B, int E, typename F> __device__ __forceinline__ bool steps(int left, F &&step) {
    step(std::integral_constant<int, B>{});
    if (left == B + 1) return true;
    if constexpr (B + 1 < E) return steps<B + 1, E>(left, step);
    return false;
}

// WGM x WGN waves of MT x NT tiles of 16 x 16: a workgroup's outputs are BM x BN.  K is
// staged 64 at a time by direct global -> LDS loads, a block a wave and load, into NB
// buffers, each stage's loads issued NB stages before its products.  Each buffer is its
// own array, and the stage barrier a bare s_barrier behind a wait for the next stage's
// loads only.  Past the last stage the last one is loaded again, so that the waits are
// the same for every stage; blocks past the last are the last again.  A stage's A
// fragments are read behind that barrier, before the products of the stage before; the W
// fragments of column tile j as soon as the products with the last ones are issued.
// Bound (32768 x 6144 x 2048, 2240 TOPS, 45 % of the matrix cores' dense rate at the
// clock they have then) by the stages' barriers and the latency of their loads: two
// workgroups a CU of 256 x 128, whose stores one hides behind the other's products.
template <int ACT, int MT, int NT, int WGM, int WGN, int NB>
__global__ __launch_bounds__(WGM *WGN *kWave, NB == 4 ? 1 : MT * NT == 32 ? 2 : 3) void dense_int8_kernel(Int8GemmArgs g) {
    using A = Act<ACT>;
    constexpr int BM = 16 * MT * WGM, BN = 16 * NT * WGN, BK = 64, kWaves = WGM * WGN;
    constexpr int kBlocksA = BM / 16 / kWaves, kBlocksW = BN / 16 / kWaves, kLoads = kBlocksA + kBlocksW;
    static_assert(kBlocksA * 16 * kWaves == BM && kBlocksW * 16 * kWaves == BN, "whole blocks a wave");
    __shared__ __attribute__((aligned(16))) int8_t A0[BM * BK], A1[BM * BK], A2[BM * BK], A3[NB > 3 ? BM * BK : 16];
    __shared__ __attribute__((aligned(16))) int8_t W0[BN * BK], W1[BN * BK], W2[BN * BK], W3[NB > 3 ? BN * BK : 16];

    const int tiles_m = (int)((g.M + BM - 1) / BM), tiles_n = (int)((g.N + BN - 1) / BN);
    const int nwg = tiles_m * tiles_n;
    constexpr int GM = 4;
    int id = blockIdx.x;
    // A contiguous range of tiles for each XCD.  (Other numbers of tiles stay in order: the
    // rows' tiles of one column then lie on several XCDs, and each fetches its weights again.
    // 320 x 32003 x 2048, 753 tiles: 205 MB read where 66 are needed, at the copy's rate.)
    if (nwg % 8 == 0) id = (id % 8) * (nwg / 8) + id / 8;
    const int group = id / (GM * tiles_n);
    const int first_m = group * GM;
    const int gm = (tiles_m - first_m < GM) ? tiles_m - first_m : GM;
    const int in_group = id - group * GM * tiles_n;
    const int64_t m0 = (int64_t)(first_m + in_group % gm) * BM, n0 = (int64_t)(in_group / gm) * BN;

    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = w % WGM, wn = w / WGM;
    const int stages = (int)((g.K + BK - 1) / BK);

    // the wave's blocks of 16 rows (the last one again past the end) and the lane's 16 bytes
    const int8_t *pa[kBlocksA], *pw[kBlocksW];
#pragma unroll
    for (int h = 0; h < kBlocksA; ++h) {
        const int64_t row = m0 + 16 * (kBlocksA * w + h);
        pa[h] = g.A + block_of(row < g.M ? row : g.M - 1, g.K);
    }
#pragma unroll
    for (int h = 0; h < kBlocksW; ++h) {
        const int64_t row = n0 + 16 * (kBlocksW * w + h);
        pw[h] = g.W + block_of(row < g.N ? row : g.N - 1, g.K);
    }
    auto bufs = [&](auto bc) {
        constexpr int b = decltype(bc)::value;
        int8_t *a = b == 0 ? A0 : b == 1 ? A1 : b == 2 ? A2 : A3;
        int8_t *ww = b == 0 ? W0 : b == 1 ? W1 : b == 2 ? W2 : W3;
        return std::make_pair(a, ww);
    };
    auto issue = [&](int8_t *as, int8_t *ws, int stage) {
        const uint32_t at = (uint32_t)(stage < stages ? stage : stages - 1) * 1024u + 16u * lane;
#pragma unroll
        for (int h = 0; h < kBlocksA; ++h)
            __builtin_amdgcn_global_load_lds(reinterpret_cast<const void *>(pa[h] + at),
                                             &as[16 * (kBlocksA * w + h) * BK], 16, 0, 0);
#pragma unroll
        for (int h = 0; h < kBlocksW; ++h)
            __builtin_amdgcn_global_load_lds(reinterpret_cast<const void *>(pw[h] + at),
                                             &ws[16 * (kBlocksW * w + h) * BK], 16, 0, 0);
    };
    const int mine = place(lane % 16, lane / 16);
    auto frag = [&](const int8_t *buf, int row0) { return *reinterpret_cast<const uint4 *>(&buf[row0 * BK + mine]); };
    uint4 af[2][MT], wf[NT];
    i32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    // (an s_waitcnt immediate: vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8)
    auto stage_barrier = [&](auto vc) {
        constexpr int v = decltype(vc)::value;
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt((v & 15) | (v >> 4) << 14 | (0x7 << 4));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    };
    issue(A0, W0, 0);
    issue(A1, W1, 1);
    issue(A2, W2, 2);
    if constexpr (NB > 3) issue(A3, W3, 3);
    stage_barrier(std::integral_constant<int, kLoads * (NB - 1)>{});
#pragma unroll
    for (int i = 0; i < MT; ++i) af[0][i] = frag(A0, 16 * (MT * wm + i));
#pragma unroll
    for (int j = 0; j < NT; ++j) wf[j] = frag(W0, 16 * (NT * wn + j));
    // the W fragment is the first operand, so the C tiles are held transposed: lane l
    // holds row 16 i + l % 16, columns 16 j + 4 (l / 16) .. + 3
    // (The loop is left right behind the last stage: where that one could be followed by
    // another turn, the compiler waits for all loads in flight before a stage's reads, as
    // it still does once a turn.  256 x 128 outputs of 32768 x 6144 x 2048: 454 us with
    // such waits, 422 with one in two turns of NB stages, 419 in four.)
    constexpr int kTurn = 4 * NB;
    for (int s0 = 0;; s0 += kTurn) {
        const bool done = steps<0, kTurn>(stages - s0, [&](auto sc) {
            constexpr int b = decltype(sc)::value, cur = b % 2, next = (b + 1) % NB;
            stage_barrier(std::integral_constant<int, kLoads * (NB - 2)>{});
            const auto here = bufs(std::integral_constant<int, b % NB>{}), ahead = bufs(std::integral_constant<int, next>{});
            issue(here.first, here.second, s0 + b + NB);
            const int8_t *as = ahead.first, *ws = ahead.second;
#pragma unroll
            for (int i = 0; i < MT; ++i) af[1 - cur][i] = frag(as, 16 * (MT * wm + i));
            #pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i][j] = mfma_i8(wf[j], af[cur][i], acc[i][j]);
                wf[j] = frag(ws, 16 * (NT * wn + j));
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        if (done) break;
    }

    const int64_t row0 = m0 + 16 * MT * wm, col0 = n0 + 16 * NT * wn;
    float sa[MT], sw[NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = row0 + 16 * i + lane % 16;
        sa[i] = g.a_scale[m < g.M ? m : g.M - 1];
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t n = col0 + 16 * j + 4 * (lane / 16) + e;
            sw[j][e] = g.w_scale[n < g.N ? n : g.N - 1];
        }
    // Through the LDS: each wave writes its tile, a part at a time, into one of the stage
    // arrays and reads it back as whole rows, so that a store writes rows' neighbouring
    // columns.  Chunk c of 16 bytes is at c ^ (row % chunks).  (Stored from the registers,
    // float32 rows of odd length took 36 us of 419 x 23331 x 266, now 22.)
    constexpr int kCols = 16 * NT, EB = A::kBytes, E = 16 / EB, kChunks = kCols / E, kStage = (BM < BN ? BM : BN) * BK;
    constexpr int kPart = MT * 16 * kCols * EB <= kStage ? MT : kStage / (16 * kCols * EB);  // row tiles at once
    static_assert(kPart > 0 && MT % kPart == 0 && (NB > 3 ? kWaves <= 8 : kWaves <= 4), "a part of a wave's tile in a stage array");
    using T = typename A::T;
    __builtin_amdgcn_s_waitcnt(0);  // the loads past the last stage
    __syncthreads();
    int8_t *stage = w == 0 ? A0 : w == 1 ? A1 : w == 2 ? A2 : w == 3 ? W0 : w == 4 ? W1 : w == 5 ? W2 : w == 6 ? W3 : A3;
    T *ob = reinterpret_cast<T *>(stage);
    auto place_in = [&](int row, int c) { return row * kCols + E * (c ^ (row % kChunks)); };
    const bool pieces = g.ldc % E == 0 && reinterpret_cast<uintptr_t>(g.C) % 16 == 0 && col0 + kCols <= g.N;
#pragma unroll
    for (int i0 = 0; i0 < MT; i0 += kPart) {
#pragma unroll
        for (int i = i0; i < i0 + kPart; ++i) {
            const int row = 16 * (i - i0) + lane % 16;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (float)acc[i][j][e] * sa[i] * sw[j][e];
                if constexpr (ACT == kF32)
                    *reinterpret_cast<float4 *>(&ob[place_in(row, 4 * j + lane / 16)]) = make_float4(y[0], y[1], y[2], y[3]);
                else
                    *reinterpret_cast<uint2 *>(&ob[place_in(row, 2 * j + lane / 32) + 4 * (lane / 16 % 2)]) =
                        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            }
        }
        const int64_t first = row0 + 16 * i0;
        T *C = static_cast<T *>(g.C) + first * g.ldc + col0;
        if (pieces) {
            constexpr int kRows = kWave / kChunks;  // rows of a store
#pragma unroll
            for (int t = 0; t < 16 * kPart / kRows; ++t) {
                const int row = kRows * t + lane / kChunks, chunk = lane % kChunks;
                const uint4 v = *reinterpret_cast<const uint4 *>(&ob[place_in(row, chunk)]);
                if (first + row < g.M) *reinterpret_cast<uint4 *>(C + (int64_t)row * g.ldc + E * chunk) = v;
            }
        } else {
            constexpr int kAcross = kCols < kWave ? kCols : kWave, kRows = kWave / kAcross;
#pragma unroll 8
            for (int t = 0; t < 16 * kPart / kRows; ++t) {
                const int row = kRows * t + lane / kAcross;
                if (first + row >= g.M) continue;
#pragma unroll
                for (int c = lane % kAcross; c < kCols; c += kAcross)
                    if (col0 + c < g.N) C[(int64_t)row * g.ldc + c] = ob[place_in(row, c / E) + c % E];
            }
        }
    }
}

// ------------------------------------------------------------------ products, few rows

// Up to 16 MT rows: the weights are read once, by waves that each take a share of K of
// 16 output channels, 8 steps of 64 in flight; the waves' sums join in the LDS.
template <int ACT, int MT, int W>
__global__ __launch_bounds__(W *kWave) void dense_int8_few_kernel(Int8GemmArgs g) {
    using A = Act<ACT>;
    constexpr int kSteps = 8;
    __shared__ i32x4 sums[W][MT][kWave];
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane % 16, c = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int mine = place(r, c);
    const int steps = (int)((g.K + 63) / 64), share = (steps + W - 1) / W;
    const int first = w * share, last = first + share < steps ? first + share : steps;
    const int8_t *pw = g.W + block_of(n0, g.K) + mine, *pa[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) pa[i] = g.A + block_of(16 * i < g.M ? 16 * i : g.M - 1, g.K) + mine;
    i32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = i32x4{0, 0, 0, 0};
    for (int s = first; s < last; s += kSteps) {
        uint4 wf[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int64_t at = 1024 * (int64_t)(s + k < last ? s + k : last - 1);
            wf[k] = *reinterpret_cast<const uint4 *>(pw + at);
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            if (s + k >= last) break;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = mfma_i8(wf[k], *reinterpret_cast<const uint4 *>(pa[i] + 1024 * (int64_t)(s + k)), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sums[w][i][lane] = acc[i];
    __syncthreads();
    for (int i = w; i < MT; i += W) {
        i32x4 t = sums[0][i][lane];
#pragma unroll
        for (int k = 1; k < W; ++k) t += sums[k][i][lane];
        const int64_t m = 16 * i + r;
        if (m >= g.M) continue;
        const float sa = g.a_scale[m];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t col = n0 + 4 * c + e;
            if (col < g.N) A::st(static_cast<typename A::T *>(g.C) + m * g.ldc + col, (float)t[e] * sa * g.w_scale[col]);
        }
    }
}

// The same for up to kFusedRows rows of up to kFusedK inputs that the outputs do not
// overwrite, which every workgroup brings to 8 bits itself while its weights are on their
// way: wave w takes rows w and w + 4 into the LDS.
//
// The limits, by measurements at 200 sizes with weights from HBM.  us of the GPU alone, in
// two launches and in one; in brackets of a call from Python, at least 9.2 in two and 6.9
// in one:
//   2048 x 2048: 1 row 7.0, 4.9; 8 rows 7.5, 7.2; 12 rows (a copy of this for 16) 7.8, 9.6.
//   4096 inputs (a copy): 1 row 10.4, 7.0; 8 rows 11.1, 13.0; and its registers make 2048
//   inputs slower, 8 rows 8.2.
//   8192 outputs, two workgroups a CU, of 2048 inputs: 4 rows 8.6, 7.5 (8.9, 7.4); 8 rows
//   8.7, 9.9 (8.9, 9.9), the worst below that limit.
//   16384 outputs, four workgroups a CU, as many as it holds: 8 rows of 512 6.9, 8.2 (9.5,
//   8.1); 4 of 2048 10.5, 9.8 (10.3, 9.8); 8 of 2048 10.6, 13.0 (10.4, 12.9).
//   32003: 1 row of 512 7.9, 10.9 (9.5, 10.7); 8 rows of 2048 15.9, 21.6 (15.6, 21.3): every
//   turn of workgroups brings the rows to 8 bits again.
constexpr int kFusedRows = 8, kFusedK = 2048;

bool in_one_launch(const Int8GemmArgs &g) {
    return g.M <= kFusedRows && g.K <= kFusedK && (g.N <= 8192 || (g.N <= 16384 && g.M * g.K <= 8192));
}

template <int ACT, int OUT>
__global__ __launch_bounds__(256) void dense_int8_fused_kernel(QuantArgs a, Int8GemmArgs g) {
    using O = Act<OUT>;
    constexpr int W = 4, kSteps = kFusedK / 64 / W, EB = Act<ACT>::kBytes, E = 16 / EB;
    constexpr int N = kFusedK / (E * kWave), kTurns = kFusedRows / W;
    __shared__ __attribute__((aligned(16))) int8_t rows[kFusedK * 16];
    __shared__ i32x4 sums[W][kWave];
    __shared__ float scales[kFusedRows];
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane % 16, c = lane / 16, K = (int)g.K, M = (int)g.M;
    const int steps = (K + 63) / 64, share = (steps + W - 1) / W;
    const int first = w * share, last = first + share < steps ? first + share : steps;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int mine = place(r, c);
    const int8_t *pw = g.W + block_of(n0, g.K) + mine;
    uint4 wf[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k)  // (past the share: the last step's, not used)
        wf[k] = *reinterpret_cast<const uint4 *>(pw + 1024 * (int64_t)(first + k < steps ? first + k : steps - 1));
    u32x4 piece[kTurns][N];
    bool again[kTurns];
    uint32_t top[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const int m = w + W * t;
        load_row<ACT>(static_cast<const unsigned char *>(a.x) + (m < M ? m * a.ldx * EB : 0), m < M ? K : 0, lane, kWave, piece[t]);
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const int m = w + W * t;
        again[t] = false;
        if (m >= M) continue;
        RowStat s{0, 0.0f};
        take_row<ACT>(s, piece[t]);
        s = joined<1>(s);
        put_row<ACT>(rows, m, 64 * steps, lane, kWave, piece[t], s);
        if (lane == 0) scales[m] = row_scale(a, s);
        again[t] = sum_again(a, s);
        top[t] = (uint32_t)__builtin_amdgcn_readfirstlane((int)s.top);
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
        if (__builtin_expect(again[t], 0)) {
            const float scale = row_scale_again<ACT, 1>(a, w + W * t, top[t]);
            if (lane == 0) scales[w + W * t] = scale;
        }
    __syncthreads();
    i32x4 acc = {0, 0, 0, 0};  // (rows that are none hold anything, and are not stored)
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
        if (first + k < last) acc = mfma_i8(wf[k], *reinterpret_cast<const uint4 *>(&rows[1024 * (first + k) + mine]), acc);
    sums[w][lane] = acc;
    __syncthreads();
    if (w > 0 || r >= M) return;
#pragma unroll
    for (int k = 1; k < W; ++k) acc += sums[k][lane];
    const float sa = scales[r];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t col = n0 + 4 * c + e;
        if (col < g.N) O::st(static_cast<typename O::T *>(g.C) + r * g.ldc + col, (float)acc[e] * sa * g.w_scale[col]);
    }
}

template <int ACT, int MT, int NT, int WGM, int WGN, int NB> void launch_tiles(const Int8GemmArgs &g, hipStream_t stream) {
    constexpr int BM = 16 * MT * WGM, BN = 16 * NT * WGN;
    const dim3 grid((unsigned)((g.M + BM - 1) / BM * ((g.N + BN - 1) / BN)));
    dense_int8_kernel<ACT, MT, NT, WGM, WGN, NB><<<grid, WGM * WGN * kWave, 0, stream>>>(g);
}

// By rows and numbers of tiles, from measurements at 3 x 9 x 17 sizes (K = 512 to 8192):
// up to 32 rows the weights are streamed (6144 x 2048, 32 rows: 6.9 us, 7.2 in tiles of
// 64 x 64; 33 rows 9.0, 7.1); then the smallest tiles of which three a CU are enough
// (320 x 6144 x 2048: 10.2 us with 64 x 64, 12.4 with 128 x 128, 18.6 with 256 x 128;
// 2048 x 6144 x 2048: 48, 28.7, 29.7), else 256 x 128, or 256 x 256 where K is long
// (8192 x 8192 x 8192: 404 us against 428, 2720 TOPS; 16384 x 6144 x 512: 90, 78).
template <int ACT> void launch_product(const Int8GemmArgs &g, hipStream_t stream) {
    const dim3 few((unsigned)((g.N + 15) / 16));
    if (g.M <= 16) return dense_int8_few_kernel<ACT, 1, 4><<<few, 4 * kWave, 0, stream>>>(g);
    if (g.M <= 32) return dense_int8_few_kernel<ACT, 2, 4><<<few, 4 * kWave, 0, stream>>>(g);
    auto tiles = [&](int64_t bm, int64_t bn) { return ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn); };
    if (tiles(64, 64) <= 768) return launch_tiles<ACT, 2, 2, 2, 2, 4>(g, stream);
    if (tiles(128, 128) <= 768) return launch_tiles<ACT, 4, 4, 2, 2, 3>(g, stream);
    if (g.K >= 4096) return launch_tiles<ACT, 8, 4, 2, 4, 4>(g, stream);
    launch_tiles<ACT, 8, 4, 2, 2, 3>(g, stream);
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs &a, hipStream_t stream) {
    if (a.act == kBF16) launch_quantize<kBF16>(a, stream);
    else launch_quantize<kF32>(a, stream);
    return hipGetLastError();
}

hipError_t launch_dense_int8_rows(const QuantArgs &a, const Int8GemmArgs &g, bool apart, hipStream_t stream) {
    if (apart && in_one_launch(g)) {
        const dim3 grid((unsigned)((g.N + 15) / 16));
        if (a.act == kBF16 && g.act == kBF16) dense_int8_fused_kernel<kBF16, kBF16><<<grid, 256, 0, stream>>>(a, g);
        else if (a.act == kBF16) dense_int8_fused_kernel<kBF16, kF32><<<grid, 256, 0, stream>>>(a, g);
        else if (g.act == kBF16) dense_int8_fused_kernel<kF32, kBF16><<<grid, 256, 0, stream>>>(a, g);
        else dense_int8_fused_kernel<kF32, kF32><<<grid, 256, 0, stream>>>(a, g);
        return hipGetLastError();
    }
    const hipError_t e = launch_quantize_rows(a, stream);
    return e != hipSuccess ? e : launch_dense_int8(g, stream);
}

hipError_t launch_dense_int8(const Int8GemmArgs &g, hipStream_t stream) {
    if (g.act == kBF16) launch_product<kBF16>(g, stream);
    else launch_product<kF32>(g, stream);
    return hipGetLastError();
}

}  // namespace hm
