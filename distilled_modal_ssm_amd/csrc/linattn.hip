// linattn.hip -- linear attention with a decay: the recurrence over a prompt
// and for one generated token.  Per batch row and head, S [dk][dv]:
//     S_t = exp(a_t) S_{t-1} + k_t v_t^T,      y_t = scale * S_t^T q_t.
//
// Prompt.  In chunks of C tokens, with S the state entering the chunk, G_t the
// sum of a up to and with token t of the chunk, and E = G at the chunk's end:
//     y_t = scale ( exp(G_t) S^T q_t + sum_{s<=t} exp(G_t - G_s) (q_t . k_s) v_s )
//     S'  = exp(E) S + sum_s k_s (exp(E - G_s) v_s)^T
// which are four products on the matrix cores: K Q^T (C x C), the weighted
// result times V, S^T Q^T, and K^T V with V weighted.  All exponents are of
// sums over later tokens, at most 0 where a is, so nothing overflows.
//
// Precision.  bfloat16 parts of operands, float32 accumulation, 16x16x32 MFMAs:
//   q, k, v      one part (bfloat16) or three (float32: 24 bits);
//   weighted V   three parts, for both types: the state keeps float32 precision
//                over any length;
//   S, weighted K Q^T  as operands of y only: three parts (float32), one
//                (bfloat16: each adds a rounding like that of y itself, so y's
//                error is at most 1.41 of the one its own rounding makes);
//   products of parts i and j are left out where i + j > 2 (below 2^-24).
// G is summed in float64 (and in units of log 2, for the exponential's
// instruction).  The rounding of the state's factor exp(E) is made good in the
// next chunk's: a head that forgets slowly multiplies by the same factor over and
// over, so its rounding would add up.
//
// Workgroup: a batch row, a head and 64 value columns, 16 a wave.  The wave's
// part of the state, [dk][16], stays in the accumulators of the K^T V products
// from chunk to chunk (lane = value column, registers = key rows).  The key rows
// of an MFMA tile are chosen so that two tiles' registers are, converted in
// place, the S^T operand of the next chunk (lane group g: key rows 8g .. 8g+7 of
// each 32): the state never passes through the LDS.  K and V come out of the LDS
// transposed (ds_read_b64_tr_b16).
//
// A prompt of too few rows and heads to fill the GPU is cut into segments of
// chunks: the state-only form of the kernel runs over every segment but the last
// from a zero state (k and v only), a scan joins the states, and the full form
// starts every segment from its own.
#include "hm_internal.hpp"

#include <type_traits>

namespace hm {
namespace {

constexpr int kThreads = 256;

// exp(a) of a log decay; a is bounded below so that sums of it stay finite
__device__ __forceinline__ float bound_decay(float a) { return a < -1000.f ? -1000.f : a; }

// ------------------------------------------------------------------ prompt

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// c[n] += a[n] b[n] for N tiles: the products of their parts i and j, i + j
// decreasing so that the smallest come first, tile after tile in between (a
// product that waits for the one before of its own tile leaves a gap).
template <int N, int NA, int NB, int MA, int MB>
__device__ __forceinline__ void mfma_tiles(const uint4 (&a)[MA][NA], const uint4 (&b)[MB][NB], f32x4 *c) {
    constexpr int P = NA > NB ? NA : NB;
#pragma unroll
    for (int sum = P - 1; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = sum - i;
            if (j < 0 || j >= NB) continue;
#pragma unroll
            for (int n = 0; n < N; ++n)
                c[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[n][i]),
                                                               __builtin_bit_cast(bf16x8, b[n][j]), c[n], 0, 0, 0);
        }
}

// x, y -> their leading bfloat16 parts packed; x, y become what is left.
__device__ __forceinline__ uint32_t take_part(float &x, float &y) {
    const uint32_t w = pack_bf16x2(x, y);
    x -= bf16_lo(w);
    y -= bf16_hi(w);
    return w;
}

template <int N>
__device__ __forceinline__ void split8(float (&x)[8], uint4 (&out)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
        out[n] = make_uint4(take_part(x[0], x[1]), take_part(x[2], x[3]), take_part(x[4], x[5]), take_part(x[6], x[7]));
}

// 16 bytes of a row from column c on, of n columns (zero past them).  G: bytes
// that every address and the row's width are a multiple of (16, 8 or an element).
template <int ACT, int G>
__device__ __forceinline__ uint4 load_piece(const typename Act<ACT>::T *row, int c, int n) {
    constexpr int EB = Act<ACT>::kBytes, PER = 16 / EB;
    uint4 w = make_uint4(0, 0, 0, 0);
    if constexpr (G == 16) {
        if (c < n) w = *reinterpret_cast<const uint4 *>(row + c);
    } else if constexpr (G == 8) {
        if (c < n) {
            const uint2 x = *reinterpret_cast<const uint2 *>(row + c);
            w.x = x.x;
            w.y = x.y;
        }
        if (c + PER / 2 < n) {
            const uint2 x = *reinterpret_cast<const uint2 *>(row + c + PER / 2);
            w.z = x.x;
            w.w = x.y;
        }
    } else {
        uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (c + e < n) {
                if constexpr (EB == 2)
                    x[e / 2] |= (uint32_t)row[c + e] << (16 * (e & 1));
                else
                    x[e] = __float_as_uint(row[c + e]);
            }
        w = make_uint4(x[0], x[1], x[2], x[3]);
    }
    return w;
}

// A piece into its place in the parts' LDS planes.
template <int ACT, int PLANE>
__device__ __forceinline__ void store_piece(uint16_t *at, const uint4 w) {
    if constexpr (ACT == kBF16) {
        *reinterpret_cast<uint4 *>(at) = w;
    } else {
        float x = __uint_as_float(w.x), y = __uint_as_float(w.y), z = __uint_as_float(w.z), u = __uint_as_float(w.w);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            const uint32_t lo = take_part(x, y);
            *reinterpret_cast<uint2 *>(at + n * PLANE) = make_uint2(lo, take_part(z, u));
        }
    }
}

// Four rows of 16 columns of a plane, transposed: lane i of a group of 16 gets
// column i.  Each lane names 4 columns of a row: lanes 4j .. 4j+3 row j.
__device__ __forceinline__ uint2 read_transposed(const uint16_t *at) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at));
}

__device__ __forceinline__ uint4 load_bounded(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

constexpr int kVT = 64;  // value columns of a workgroup

struct LinAttnPlan {
    int64_t segs, seg_chunks;   // segments of the prompt, and chunks of each
    int chunk;                  // tokens of a chunk
    int vtiles;                 // workgroups of a row and head
    size_t off_decay, bytes;    // float [B H][segs][dk][dv] states; float2 [B H][segs] segment factors
};

template <int ACT, int DK> struct ChunkGeom {
    static constexpr int C = (ACT == kBF16 && DK <= 128) ? 64 : 32;
    static constexpr int NP = ACT == kBF16 ? 1 : 3;  // parts of q, k, v, and of what y's products round
    static constexpr int EB = Act<ACT>::kBytes;
    // LDS rows in elements, by the counted conflicts of each access (cycles beyond
    // the first ones of a wave's instruction): Q, read in rows of 16 bytes, has none
    // where the row is an odd multiple of 16 elements (4 at DK + 8); K is read more
    // often transposed, with 2 where its row is an odd multiple of 32 (4 to 6 else).
    static constexpr int QS = DK + 16;
    static constexpr int KS = DK == 32 ? 32 : DK + 32;
    static constexpr int VS = kVT + 8, PS = C + 8;
    static constexpr int QP = C * QS, KP = C * KS, VP = C * VS, PP = C * PS;  // planes
    static constexpr int kBytes = 2 * NP * (QP + KP + VP + PP) + 2 * (C * 16 + 4) + 8;
    static constexpr int kPerCU = kBytes <= 80 * 1024 ? 2 : 1;
};

template <int ACT, int DK, int G, bool FULL>
__global__ __launch_bounds__(kThreads, (ChunkGeom<ACT, DK>::kPerCU)) void linattn_chunk_kernel(LinAttnArgs a, LinAttnPlan p) {
    using T = typename Act<ACT>::T;
    using M = ChunkGeom<ACT, DK>;
    constexpr int C = M::C, NP = M::NP, PER = 16 / M::EB;
    constexpr int RP = DK / PER, NQ = C * RP / kThreads, RSTEP = kThreads / RP;     // q, k pieces of a row, a thread
    constexpr int VP = kVT / PER, NV = C * VP / kThreads, VSTEP = kThreads / VP;    // v pieces
    constexpr int TT = C / 16, KK = C / 32, PAIRS = DK / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    uint16_t *Qs = reinterpret_cast<uint16_t *>(smem), *Ks = Qs + NP * M::QP, *Vs = Ks + NP * M::KP,
             *Ps = Vs + NP * M::VP;
    double *Gs = reinterpret_cast<double *>(Ps + NP * M::PP);  // [2][C] by the chunk's parity, as the next three
    float *from_start = reinterpret_cast<float *>(Gs + 2 * C), *to_end = from_start + 2 * C, *factor = to_end + 2 * C;

    // neighbouring value tiles of a head and segment on one XCD (workgroups go
    // round the eight by their index): they read the same q and k
    const int64_t units = a.s.B * a.s.H * p.segs;
    const int64_t local = blockIdx.x >> 3, unit = local / p.vtiles * 8 + (blockIdx.x & 7);
    if (unit >= units) return;
    const int vt = (int)(local % p.vtiles);
    const int64_t bh = unit / p.segs, seg = unit - bh * p.segs, b = bh / a.s.H, h = bh - b * a.s.H;
    if (!FULL && seg == p.segs - 1) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), li = lane & 15,
              lg = lane >> 4;
    const int dk = a.s.dk, dv = a.s.dv, v0 = vt * kVT, vcols = dv - v0 < kVT ? dv - v0 : kVT;
    int64_t len = a.L;
    if (a.lengths) len = a.lengths[b] < 0 ? 0 : a.lengths[b] < a.L ? a.lengths[b] : a.L;
    const int64_t begin = seg * p.seg_chunks * C, end = begin + p.seg_chunks * C < a.L ? begin + p.seg_chunks * C : a.L;
    const int64_t rows = len <= begin ? 0 : (len < end ? len : end) - begin;  // tokens of this segment

    const T *q = static_cast<const T *>(a.q) + (b * a.L + begin) * a.ld_q + h * a.s.qh / a.s.H * dk;
    const T *k = static_cast<const T *>(a.k) + (b * a.L + begin) * a.ld_k + h * a.s.kh / a.s.H * dk;
    const T *v = static_cast<const T *>(a.v) + (b * a.L + begin) * a.ld_v + h * a.s.vh / a.s.H * dv + v0;
    T *y = static_cast<T *>(a.y) + (b * a.L + begin) * a.ld_y + h * dv + v0;
    const float *decay = a.decay ? a.decay + (a.ld_decay ? (b * a.L + begin) * a.ld_decay : 0) + h : nullptr;
    const int64_t cells = (int64_t)dk * dv;

    // the state: tile 2P + u, register r = key row 32 P + 8 lg + 4 u + r, value column li of the wave
    const int col = 16 * wave + li;
    f32x4 S[2 * PAIRS];
    {
        const float *from = nullptr;
        if (FULL) {
            if (p.segs > 1)
                from = reinterpret_cast<const float *>(a.ws) + (bh * p.segs + seg) * cells;
            else if (a.state_in)
                from = a.state_in + bh * cells;
        }
#pragma unroll
        for (int t = 0; t < 2 * PAIRS; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * (t & ~1) + 8 * lg + 4 * (t & 1) + r;
                S[t][r] = from && row < dk && col < vcols ? from[(int64_t)row * dv + v0 + col] : 0.f;
            }
    }

    // tokens of the next chunk, on their way
    const int qr = tid / RP, qc = tid % RP * PER, vr = tid / VP, vc = tid % VP * PER;
    uint4 rq[NQ], rk[NQ], rv[NV];
    auto fetch = [&](int64_t t0) {
        const int64_t n = rows - t0;
        if constexpr (G == 16) {
            // rows and columns past the end read as zero by the bounds of the buffer
            const uint32_t last = n <= 0 ? 0 : (uint32_t)(n < C ? n - 1 : C - 1);
            const uint32_t sq = (uint32_t)a.ld_q * M::EB, sk = (uint32_t)a.ld_k * M::EB, sv = (uint32_t)a.ld_v * M::EB;
            const auto bq = make_region(q + t0 * a.ld_q, n <= 0 ? 0 : last * sq + dk * M::EB);
            const auto bk = make_region(k + t0 * a.ld_k, n <= 0 ? 0 : last * sk + dk * M::EB);
            const auto bv = make_region(v + t0 * a.ld_v, n <= 0 ? 0 : last * sv + vcols * M::EB);
            const uint32_t oc = qc < dk ? qc * M::EB : 0x80000000u, ov = vc < vcols ? vc * M::EB : 0x80000000u;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                if (FULL) rq[i] = load_bounded(bq, oc + (qr + i * RSTEP) * sq);
                rk[i] = load_bounded(bk, oc + (qr + i * RSTEP) * sk);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) rv[i] = load_bounded(bv, ov + (vr + i * VSTEP) * sv);
        } else {
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int r = qr + i * RSTEP;
                rq[i] = rk[i] = make_uint4(0, 0, 0, 0);
                if (r < n) {
                    if (FULL) rq[i] = load_piece<ACT, G>(q + (t0 + r) * a.ld_q, qc, dk);
                    rk[i] = load_piece<ACT, G>(k + (t0 + r) * a.ld_k, qc, dk);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int r = vr + i * VSTEP;
                rv[i] = make_uint4(0, 0, 0, 0);
                if (r < n) rv[i] = load_piece<ACT, G>(v + (t0 + r) * a.ld_v, vc, vcols);
            }
        }
    };
    // The last wave, which has the fewest K Q^T tiles, forms a chunk's decays while
    // the chunk before is worked on.  `error`: the state's factor as it should be
    // over what float32 made of it, handed on to the next chunk's factor, so that
    // the factors' product over many chunks is right to a rounding.
    float ra = 0.f;
    double total = 0.0, error = 1.0;
    auto fetch_decay = [&](int64_t t0) {
        ra = 0.f;
        if (decay && lane < C && t0 + lane < rows) ra = bound_decay(decay[(t0 + lane) * a.ld_decay]);
    };
    auto form_decays = [&](int at) {
        constexpr double kLog2e = 1.4426950408889634074;
        double g = ra * kLog2e;
#pragma unroll
        for (int d = 1; d < C; d <<= 1) {
            const double o = __shfl_up(g, d);
            if (lane >= d) g += o;
        }
        const double e = __shfl(g, C - 1);
        total += e;
        if (lane < C) {
            Gs[at * C + lane] = g;
            from_start[at * C + lane] = __builtin_amdgcn_exp2f((float)g);
            to_end[at * C + lane] = __builtin_amdgcn_exp2f((float)(e - g));
        }
        const double f = exp2(e) * error;
        const float ff = (float)f;
        error = ff > 1e-30f ? f / (double)ff : 1.0;
        if (lane == 0) factor[at] = ff;
    };

    // tiles above the diagonal that the products read: zero, once
    if (FULL)
        for (int i = tid; i < NP * M::PP; i += kThreads) Ps[i] = 0;
    fetch(0);
    if (wave == 3) {
        fetch_decay(0);
        form_decays(0);
        fetch_decay(C);
    }
    for (int64_t t0 = 0, odd = 0; t0 < rows; t0 += C, odd ^= 1) {
        __syncthreads();  // the chunk before is done with the LDS
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if (FULL) store_piece<ACT, M::QP>(Qs + (qr + i * RSTEP) * M::QS + qc, rq[i]);
            store_piece<ACT, M::KP>(Ks + (qr + i * RSTEP) * M::KS + qc, rk[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) store_piece<ACT, M::VP>(Vs + (vr + i * VSTEP) * M::VS + vc, rv[i]);
        fetch(t0 + C);
        __syncthreads();
        if (wave == 3) {
            form_decays((int)odd ^ 1);
            fetch_decay(t0 + 2 * C);
        }
        const double *gs = Gs + odd * C;
        const float *fs = from_start + odd * C, *te = to_end + odd * C;

        f32x4 acc[TT];
        if constexpr (FULL) {
            // P[t][s] = exp(G_t - G_s) q_t . k_s for s <= t, in tiles (i, j) of 16 s x 16 t, i <= j,
            // N of them at once
            auto weigh = [&](auto count, uint32_t tiles) {
                constexpr int N = decltype(count)::value;
                const uint16_t *kat[N], *qat[N];
                f32x4 x[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t code = tiles >> (4 * n) & 15;
                    kat[n] = Ks + (16 * (code >> 2) + li) * M::KS + 8 * lg;
                    qat[n] = Qs + (16 * (code & 3) + li) * M::QS + 8 * lg;
                    x[n] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
                uint4 ka[2][N][NP], qb[2][N][NP];
                auto load = [&](int pr) {
#pragma unroll
                    for (int n = 0; n < N; ++n)
#pragma unroll
                        for (int w = 0; w < NP; ++w) {
                            ka[pr & 1][n][w] = *reinterpret_cast<const uint4 *>(kat[n] + w * M::KP + 32 * pr);
                            qb[pr & 1][n][w] = *reinterpret_cast<const uint4 *>(qat[n] + w * M::QP + 32 * pr);
                        }
                };
                load(0);
#pragma unroll
                for (int pr = 0; pr < PAIRS; ++pr) {
                    if (pr + 1 < PAIRS) load(pr + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    mfma_tiles<N>(ka[pr & 1], qb[pr & 1], x);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t code = tiles >> (4 * n) & 15;
                    const int t = 16 * (code & 3) + li, s = 16 * (code >> 2) + 4 * lg;
                    const double gt = gs[t];
                    float o[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float d = (float)(gt - gs[s + r]);
                        o[r] = x[n][r] * __builtin_amdgcn_exp2f(s + r <= t ? d : -__builtin_inff());
                    }
#pragma unroll
                    for (int w = 0; w < NP; ++w) {
                        const uint32_t lo = take_part(o[0], o[1]);
                        *reinterpret_cast<uint2 *>(Ps + w * M::PP + t * M::PS + s) = make_uint2(lo, take_part(o[2], o[3]));
                    }
                }
            };
            // codes 4 i + j of each wave's tiles; the last wave, which forms the decays, has the fewest
            constexpr uint32_t kTiles4[4] = {0xb73, 0xa62, 0xf51, 0x0}, kTiles2[4] = {0x1, 0x5, 0x0, 0x0};
            if (wave < 3)
                weigh(std::integral_constant<int, TT == 4 ? 3 : 1>{}, TT == 4 ? kTiles4[wave] : kTiles2[wave]);
            else if constexpr (TT == 4)
                weigh(std::integral_constant<int, 1>{}, kTiles4[3]);

            // exp(G_t) S^T q_t
            const uint16_t *qat = Qs + li * M::QS + 8 * lg;
            uint4 qb[2][TT][NP];
            auto load = [&](int pr) {
#pragma unroll
                for (int j = 0; j < TT; ++j)
#pragma unroll
                    for (int w = 0; w < NP; ++w)
                        qb[pr & 1][j][w] = *reinterpret_cast<const uint4 *>(qat + w * M::QP + 16 * j * M::QS + 32 * pr);
            };
            load(0);
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int pr = 0; pr < PAIRS; ++pr) {
                if (pr + 1 < PAIRS) load(pr + 1);
                __builtin_amdgcn_sched_barrier(0);
                float x[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) x[r] = S[2 * pr + r / 4][r % 4];
                uint4 sa[TT][NP];
                split8(x, sa[0]);
#pragma unroll
                for (int j = 1; j < TT; ++j)
#pragma unroll
                    for (int w = 0; w < NP; ++w) sa[j][w] = sa[0][w];
                mfma_tiles<TT>(sa, qb[pr & 1], acc);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[j] *= fs[16 * j + li];
            __syncthreads();
        }
        // V of this wave's columns as an operand: value column li, tokens 32 kk + 8 lg + 0..7
        uint4 va[KK][NP];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int w = 0; w < NP; ++w) {
                const uint16_t *at = Vs + w * M::VP + (32 * kk + 8 * lg + (li >> 2)) * M::VS + 16 * wave + 4 * (li & 3);
                const uint2 lo = read_transposed(at), hi = read_transposed(at + 4 * M::VS);
                va[kk][w] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        // K transposed, KG tiles of key rows at a time, loaded one time ahead
        constexpr int KG = NP == 3 || DK == 32 || DK == 256 ? 2 : 4, KN = KK * 2 * PAIRS / KG;
        uint4 ka[2][KG][NP];
        auto load_keys = [&](int n) {
            const int kk = n / (2 * PAIRS / KG);
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                const int t = n % (2 * PAIRS / KG) * KG + g;
#pragma unroll
                for (int w = 0; w < NP; ++w) {
                    const uint16_t *at = Ks + w * M::KP + (32 * kk + 8 * lg + (li >> 2)) * M::KS + 16 * (t & ~1) +
                                         8 * (li & 3) + 4 * (t & 1);
                    const uint2 lo = read_transposed(at), hi = read_transposed(at + 4 * M::KS);
                    ka[n & 1][g][w] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        };
        if constexpr (FULL) {
            const uint16_t *pat = Ps + li * M::PS + 8 * lg;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                uint4 pb[TT][NP], vv[TT][NP];  // tiles j from 2 kk on
#pragma unroll
                for (int j = 2 * kk; j < TT; ++j)
#pragma unroll
                    for (int w = 0; w < NP; ++w) {
                        pb[j - 2 * kk][w] = *reinterpret_cast<const uint4 *>(pat + w * M::PP + 16 * j * M::PS + 32 * kk);
                        vv[j - 2 * kk][w] = va[kk][w];
                    }
                if (kk == KK - 1) load_keys(0);
                __builtin_amdgcn_sched_barrier(0);
                if (kk == 0)
                    mfma_tiles<TT>(vv, pb, acc);
                else
                    mfma_tiles<2>(vv, pb, acc + 2 * kk);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            load_keys(0);
        }
        // the state
        const float f = factor[odd];
#pragma unroll
        for (int t = 0; t < 2 * PAIRS; ++t) S[t] *= f;
        uint4 vb[KG][3];
#pragma unroll
        for (int n = 0; n < KN; ++n) {
            const int kk = n / (2 * PAIRS / KG), first = n % (2 * PAIRS / KG) * KG;
            if (n + 1 < KN) load_keys(n + 1);
            if (first == 0) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w0 = reinterpret_cast<const uint32_t *>(&va[kk][0])[e];
                    x[2 * e] = bf16_lo(w0);
                    x[2 * e + 1] = bf16_hi(w0);
                    if constexpr (NP == 3) {
                        const uint32_t w1 = reinterpret_cast<const uint32_t *>(&va[kk][1])[e];
                        const uint32_t w2 = reinterpret_cast<const uint32_t *>(&va[kk][2])[e];
                        x[2 * e] += bf16_lo(w1) + bf16_lo(w2);
                        x[2 * e + 1] += bf16_hi(w1) + bf16_hi(w2);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= te[32 * kk + 8 * lg + e];
                split8(x, vb[0]);
#pragma unroll
                for (int g = 1; g < KG; ++g)
#pragma unroll
                    for (int w = 0; w < 3; ++w) vb[g][w] = vb[0][w];
            }
            __builtin_amdgcn_sched_barrier(0);
            mfma_tiles<KG>(ka[n & 1], vb, S + first);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (FULL) {
            const int c = 16 * wave + 4 * lg;
            T *at = y + (t0 + li) * a.ld_y + c;
            const bool whole = t0 + C <= end - begin;
#pragma unroll
            for (int j = 0; j < TT; ++j, at += 16 * a.ld_y) {
                if (c >= vcols || !(whole || t0 + 16 * j + li < end - begin)) continue;
                const f32x4 o = acc[j] * a.s.scale;
                if constexpr (G == 16 || (G == 8 && ACT == kBF16)) {
                    if constexpr (ACT == kBF16)
                        *reinterpret_cast<uint2 *>(at) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
                    else
                        *reinterpret_cast<float4 *>(at) = make_float4(o[0], o[1], o[2], o[3]);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (c + r < vcols) Act<ACT>::st(at + r, o[r]);
                }
            }
        }
    }
    if (FULL) {  // rows past the tokens
        const int64_t done = (rows + C - 1) / C * C, n = end - begin - done;
        for (int64_t i = tid; i < n * vcols; i += kThreads)
            Act<ACT>::st(y + (done + i / vcols) * a.ld_y + i % vcols, 0.f);
    }
    float *to = FULL ? a.state_out + bh * cells : reinterpret_cast<float *>(a.ws) + (bh * p.segs + seg + 1) * cells;
    if (!FULL || seg == p.segs - 1) {
#pragma unroll
        for (int t = 0; t < 2 * PAIRS; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * (t & ~1) + 8 * lg + 4 * (t & 1) + r;
                if (row < dk && col < vcols) to[(int64_t)row * dv + v0 + col] = S[t][r];
            }
    }
    if (!FULL && vt == 0 && wave == 3 && lane == 0) {
        const double f = exp2(total);
        reinterpret_cast<float2 *>(a.ws + p.off_decay)[bh * p.segs + seg] =
            make_float2((float)f, (float)(f - (double)(float)f));
    }
}

// States entering the segments: slot 0 the first state, slot s + 1 (which holds
// segment s's own end state) the state after segment s.
__global__ __launch_bounds__(kThreads) void linattn_join_kernel(LinAttnArgs a, LinAttnPlan p) {
    const int64_t cells = (int64_t)a.s.dk * a.s.dv, i = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    const int64_t bh = blockIdx.x;
    if (i >= cells) return;
    float *slot = reinterpret_cast<float *>(a.ws) + bh * p.segs * cells + i;
    const float2 *factor = reinterpret_cast<const float2 *>(a.ws + p.off_decay) + bh * p.segs;
    float x = a.state_in ? a.state_in[bh * cells + i] : 0.f;
    slot[0] = x;
    for (int64_t s = 1; s < p.segs; ++s) {
        const float2 f = factor[s - 1];
        x = fmaf(x, f.x, fmaf(x, f.y, slot[s * cells]));
        slot[s * cells] = x;
    }
}

// ------------------------------------------------------------------ one token

// One workgroup for a batch row and head: lane = value column, the four waves
// take every fourth key row.
template <int ACT>
__global__ __launch_bounds__(kThreads) void linattn_token_kernel(LinAttnArgs a) {
    using T = typename Act<ACT>::T;
    __shared__ float qs[256], ks[256], part[4][64];
    const int64_t b = blockIdx.x / a.s.H, h = blockIdx.x - b * a.s.H;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, dk = a.s.dk, dv = a.s.dv;
    int64_t src = b;
    if (a.src_rows && a.src_rows[b] >= 0 && a.src_rows[b] < a.s.B) src = a.src_rows[b];
    const float *in = a.state_in + (src * a.s.H + h) * (int64_t)dk * dv;
    float *out = a.state_out + (b * a.s.H + h) * (int64_t)dk * dv;
    const T *v = static_cast<const T *>(a.v) + b * a.ld_v + h * a.s.vh / a.s.H * dv;
    T *y = static_cast<T *>(a.y) + b * a.ld_y + h * dv;
    if (tid < dk) {
        qs[tid] = Act<ACT>::ld(static_cast<const T *>(a.q) + b * a.ld_q + h * a.s.qh / a.s.H * dk + tid);
        ks[tid] = Act<ACT>::ld(static_cast<const T *>(a.k) + b * a.ld_k + h * a.s.kh / a.s.H * dk + tid);
    }
    const float g = a.decay ? expf(bound_decay(a.decay[a.ld_decay ? b * a.ld_decay + h : h])) : 1.f;
    __syncthreads();
    for (int c0 = 0; c0 < dv; c0 += 64) {
        const int c = c0 + lane;
        float o = 0.f;
        if (c < dv) {
            const float x = Act<ACT>::ld(v + c);
            for (int i = wave; i < dk; i += 4) {
                const float s = fmaf(g, in[(int64_t)i * dv + c], ks[i] * x);
                out[(int64_t)i * dv + c] = s;
                o = fmaf(qs[i], s, o);
            }
        }
        part[wave][lane] = o;
        __syncthreads();
        if (tid < 64 && c < dv)
            Act<ACT>::st(y + c, a.s.scale * (part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid]));
        __syncthreads();
    }
}

// Padded key width, and the granule of 16, 8 bytes or an element that all rows allow.
int padded_dk(int dk) { return dk <= 32 ? 32 : dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }

LinAttnPlan linattn_plan(const LinAttnShape &s, int64_t L) {
    LinAttnPlan p;
    p.chunk = s.act == kBF16 && s.dk <= 128 ? 64 : 32;
    p.vtiles = (s.dv + kVT - 1) / kVT;
    const int64_t chunks = (L + p.chunk - 1) / p.chunk, groups = s.B * s.H * p.vtiles;
    int64_t segs = groups >= 512 ? 1 : (512 + groups - 1) / groups;
    if (segs > chunks / 8) segs = chunks / 8;
    if (segs < 1) segs = 1;
    p.seg_chunks = (chunks + segs - 1) / segs;
    p.segs = p.seg_chunks > 0 ? (chunks + p.seg_chunks - 1) / p.seg_chunks : 1;
    const size_t states = p.segs > 1 ? (size_t)(s.B * s.H * p.segs) * s.dk * s.dv * sizeof(float) : 0;
    p.off_decay = (states + 255) / 256 * 256;
    p.bytes = p.segs > 1 ? p.off_decay + (size_t)(s.B * s.H * p.segs) * sizeof(float2) : 0;
    return p;
}

int linattn_granule(const LinAttnArgs &a) {
    const int e = a.s.act == kBF16 ? 2 : 4;
    uintptr_t bits = 0;
    for (const void *x : {a.q, a.k, a.v, (const void *)a.y}) bits |= reinterpret_cast<uintptr_t>(x);
    for (int64_t n : {a.ld_q, a.ld_k, a.ld_v, a.ld_y, (int64_t)a.s.dk, (int64_t)a.s.dv}) bits |= (uintptr_t)(n * e);
    // the 16-byte loads go by 32-bit offsets from a chunk's first row
    const bool near = a.ld_q < 1 << 22 && a.ld_k < 1 << 22 && a.ld_v < 1 << 22;
    return bits % 16 == 0 && near ? 16 : bits % 8 == 0 ? 8 : e;
}

template <int ACT, int DK, int G, bool FULL>
hipError_t launch_chunks(const LinAttnArgs &a, const LinAttnPlan &p, hipStream_t stream) {
    constexpr int bytes = ChunkGeom<ACT, DK>::kBytes;
    const auto kernel = linattn_chunk_kernel<ACT, DK, G, FULL>;
    if (bytes > 65536) {
        const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (err != hipSuccess) return err;
    }
    const int64_t units = a.s.B * a.s.H * p.segs;
    kernel<<<dim3((unsigned)((units + 7) / 8 * 8 * p.vtiles)), kThreads, bytes, stream>>>(a, p);
    return hipGetLastError();
}

template <int ACT, int DK, int G>
hipError_t launch_prompt(const LinAttnArgs &a, const LinAttnPlan &p, hipStream_t stream) {
    if (p.segs > 1) {
        hipError_t err = launch_chunks<ACT, DK, G, false>(a, p, stream);
        if (err != hipSuccess) return err;
        const dim3 grid((unsigned)(a.s.B * a.s.H), (unsigned)((a.s.dk * a.s.dv + kThreads - 1) / kThreads));
        linattn_join_kernel<<<grid, kThreads, 0, stream>>>(a, p);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    return launch_chunks<ACT, DK, G, true>(a, p, stream);
}

template <int ACT, int DK>
hipError_t launch_prompt(const LinAttnArgs &a, const LinAttnPlan &p, hipStream_t stream) {
    switch (linattn_granule(a)) {
        case 16: return launch_prompt<ACT, DK, 16>(a, p, stream);
        case 8: return launch_prompt<ACT, DK, 8>(a, p, stream);
        default: return launch_prompt<ACT, DK, Act<ACT>::kBytes>(a, p, stream);
    }
}

template <int ACT>
hipError_t launch_prompt(const LinAttnArgs &a, const LinAttnPlan &p, hipStream_t stream) {
    switch (padded_dk(a.s.dk)) {
        case 32: return launch_prompt<ACT, 32>(a, p, stream);
        case 64: return launch_prompt<ACT, 64>(a, p, stream);
        case 128: return launch_prompt<ACT, 128>(a, p, stream);
        default: return launch_prompt<ACT, 256>(a, p, stream);
    }
}

}  // namespace

size_t linattn_workspace(const LinAttnShape &s, int64_t L) { return linattn_plan(s, L).bytes; }

hipError_t launch_linattn_prefill(const LinAttnArgs &a, hipStream_t stream) {
    const LinAttnPlan p = linattn_plan(a.s, a.L);
    return a.s.act == kBF16 ? launch_prompt<kBF16>(a, p, stream) : launch_prompt<kF32>(a, p, stream);
}

hipError_t launch_linattn_decode(const LinAttnArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.s.B * a.s.H));
    if (a.s.act == kBF16)
        linattn_token_kernel<kBF16><<<grid, kThreads, 0, stream>>>(a);
    else
        linattn_token_kernel<kF32><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace hm
