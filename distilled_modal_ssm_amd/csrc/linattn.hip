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
//   S, weighted K Q^T  as operands of y only: three parts (float32), two
//                (bfloat16: off by at most 2^-16 of a term, so y by 2^-16 of the
//                sum of its terms' absolute values beside its own rounding of
//                2^-8; one part: 16 x 2048 tokens, 16 heads of 128: 124 us against
//                147, but y's error is 1.41 times that of its rounding for terms
//                of random sign and has no bound where they cancel; three: 165);
//   products of parts i and j are left out where i + j > 2 (below 2^-24).
// G is summed in float64 (and in units of log 2, for the exponential's
// instruction).  The rounding of the state's factor exp(E) is made good in the
// next chunk's: a head that forgets slowly multiplies by the same factor over and
// over, so its rounding would add up.
//
// Workgroup: a batch row, a head and 64 or 128 value columns, 16 a wave.  The
// wave's part of the state, [dk][16], stays in the accumulators of the K^T V
// products from chunk to chunk (lane = value column, registers = key rows).  The
// key rows of an MFMA tile are chosen so that two tiles' registers are, converted
// in place, the S^T operand of the next chunk (lane group g: key rows 8g .. 8g+7
// of each 32): the state never passes through the LDS.  K and V come out of the
// LDS transposed (ds_read_b64_tr_b16).  Four more waves bring the next chunk.
//
// A prompt of too few rows and heads to fill the GPU is cut into segments of
// chunks: the state-only form of the kernel runs over every segment but the last
// from a zero state (k and v only, the last chunk first), a scan joins the states,
// and the full form starts every segment from its own.
//
// What bounds it (MI355X).  Many rows and heads of bfloat16: the takers' instructions,
// whose vector part (the operands' parts) and matrix part go in turn: 52 and 37 % of
// the cycles by counters; 16 rows x 2048 tokens, 16 heads of 128: 556 MB in 146-150
// us, 3.8 TB/s (a large copy has 5.4; 124 us with y's operands in one part).  A prompt
// in segments reads k and v twice (65536 tokens, 16 heads: 1.6 GB in 400 us).
// float32: the matrix cores and the vector ALUs in turn, six products of parts for
// one.  Few tokens: the two barriers and memory latency of each chunk, some 2.5 us.
//
// One token: bound by the state's way in and out (batch 256, 16 heads of 128 x 128:
// 541 MB in 102 us, 5.3 TB/s; batch 1: 4.6 us, a launch and two memory latencies).
#include "hm_internal.hpp"

#include <type_traits>

namespace hm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDk = 256;

// exp(a) of a log decay; a is bounded below so that sums of it stay finite
__device__ __forceinline__ float bound_decay(float a) { return a < -1000.f ? -1000.f : a; }

// The factor exp(a) of one token's state in two floats: a float32 one is off by up to
// 2^-24, the same way at every token, so that a head that remembers 3000 of them would
// drift by 1e-4 of its state and disagree with the prompt's.  A head that remembers more
// than eight gets 1 and exp(a) - 1, by Taylor's series (to 2^-24 of it), others exp(a)
// and nothing.
__device__ __forceinline__ float2 decay_factor(float a) {
    const float m = a * fmaf(a, fmaf(a, fmaf(a, fmaf(a, 1 / 120.f, 1 / 24.f), 1 / 6.f), 0.5f), 1.f);
    return fabsf(a) <= 0.125f ? make_float2(1.f, m) : make_float2(expf(bound_decay(a)), 0.f);
}

// f s + kv, or s + kv of a layer without decay (whose infinite states stay infinite).
template <bool DECAY>
__device__ __forceinline__ float decayed(float2 f, float s, float kv) {
    return DECAY ? fmaf(f.x, s, fmaf(f.y, s, kv)) : s + kv;
}

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

// 16 bytes at `off` of a bounded region, from column c of a row of n on: zero past
// the row's columns, and past the region's end.  G: bytes that every row and its
// width are a multiple of (16, 8 or an element).  ONCE: non-temporal, for tokens that
// are read once (six rows of up to 1501 float32 tokens, 32 heads: 103 us against 108;
// 16 x 2048 bfloat16 ones, 16 heads of 128: 150, 152; but 8 x 2000 of 32 x 32: 46, 42).
template <int ACT, int G, bool ONCE>
__device__ __forceinline__ uint4 load_piece(__amdgpu_buffer_rsrc_t region, uint32_t off, int c, int n) {
    constexpr int EB = Act<ACT>::kBytes, PER = 16 / EB;
    constexpr uint32_t kNowhere = 0x80000000u;
    constexpr int kStream = ONCE ? 2 : 0;
    if constexpr (G == 16) {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(region, c < n ? off : kNowhere, 0, kStream));
    } else if constexpr (G == 8) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b64(region, c < n ? off : kNowhere, 0, kStream);
        const auto y = __builtin_amdgcn_raw_buffer_load_b64(region, c + PER / 2 < n ? off + 8 : kNowhere, 0, kStream);
        return make_uint4(x[0], x[1], y[0], y[1]);
    } else {
        uint32_t w[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const uint32_t at = c + e < n ? off + e * EB : kNowhere;
            if constexpr (EB == 2)
                w[e] = __builtin_amdgcn_raw_buffer_load_b16(region, at, 0, 0);
            else
                w[e] = __builtin_amdgcn_raw_buffer_load_b32(region, at, 0, 0);
        }
        if constexpr (EB == 2)
            return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        else
            return make_uint4(w[0], w[1], w[2], w[3]);
    }
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

// x of the lane that a DPP control names, 0 where there is none (rows not in the mask keep 0)
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the lanes up to and with this one: within rows of 16 lanes, then the
// rows' last lanes into the rows after them.
__device__ __forceinline__ double scan_sum(double x) {
    x += dpp<0x111, 0xf>(x);  // the lane 1, 2, 4, 8 before
    x += dpp<0x112, 0xf>(x);
    x += dpp<0x114, 0xf>(x);
    x += dpp<0x118, 0xf>(x);
    x += dpp<0x142, 0xa>(x);  // lane 15 to row 1, lane 47 to row 3
    x += dpp<0x143, 0xc>(x);  // lane 31 to rows 2 and 3
    return x;
}

__device__ __forceinline__ double read_lane(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

struct LinAttnPlan {
    int64_t segs, seg_chunks;   // segments of the prompt, and chunks of each
    int chunk;                  // tokens of a chunk
    int vt, vtiles;             // value columns of a workgroup, and workgroups of a row and head
    size_t off_decay, bytes;    // float [B H][segs][dk][dv] states; float2 [B H][segs] segment factors
};

constexpr int kLds = 160 * 1024;
constexpr int kMakers = 4;  // waves that fetch, form decays and weigh K Q^T

template <int ACT, int DK, int VT> struct ChunkGeom {
    static constexpr int C = (ACT == kBF16 && DK <= 128) ? 64 : 32;
    static constexpr int NP = ACT == kBF16 ? 1 : 3;  // parts of q, k, v
    static constexpr int NS = ACT == kBF16 ? 2 : 3;  // parts of S and weighted K Q^T, as operands of y
    static constexpr int EB = Act<ACT>::kBytes;
    // LDS rows in elements, by the counted conflicts of each access (cycles beyond
    // the first ones of a wave's instruction): Q, read in rows of 16 bytes, has none
    // where the row is an odd multiple of 16 elements (4 at DK + 8); K is read more
    // often transposed, with 2 where its row is an odd multiple of 32 (4 to 6 else).
    static constexpr int QS = DK + 16;
    static constexpr int KS = DK == 32 ? 32 : DK + 32;
    static constexpr int VS = VT + 8;
    // Weighted K Q^T has C columns a row, but only 32 in its first 32 rows: later tokens'.
    // (Two workgroups of 64 bfloat16 keys and 64 value columns fit a CU with that: 128 x 16
    // heads, 16 tokens: 40 us against 67.)
    static constexpr int PS0 = 32 + 8, PS1 = C + 8;
    static constexpr int QP = C * QS, KP = C * KS, VP = C * VS, PP = 32 * PS0 + (C - 32) * PS1;  // planes
    static constexpr int buffers(int depth) {
        return 2 * (NP * depth * (QP + KP + VP) + NS * PP) + 2 * (C * 16 + 4) + 8;
    }
    // chunks in the LDS: two, or one where two do not fit
    static constexpr int kDepth = buffers(2) <= kLds ? 2 : 1;
    static constexpr int kBytes = buffers(kDepth);
    static constexpr int kTakers = VT / 16;  // waves that own value columns
    static constexpr int kThreads = 64 * (kTakers + kMakers);
    static constexpr int kWavesPerSimd = kThreads / 256;  // registers for one workgroup a CU
    static_assert(kBytes <= kLds, "LDS");
};

// The workgroup's waves have two roles.  Takers own 16 value columns each and
// hold their part of the state: they form y and the next state from what is in
// the LDS.  Makers put it there a chunk ahead: tokens (fetched a further chunk
// ahead into registers), decays, and P.  A chunk takes two steps, each ended by
// the workgroup's barrier:
//              makers                              takers
//   step 1     tokens of chunk c + 1 to the LDS    y of chunk c
//   step 2     P of chunk c + 1                    state after chunk c
template <int ACT, int DK, int VT, int G, bool FULL>
__global__ __launch_bounds__((ChunkGeom<ACT, DK, VT>::kThreads), (ChunkGeom<ACT, DK, VT>::kWavesPerSimd))
void linattn_chunk_kernel(LinAttnArgs a, LinAttnPlan p) {
    using T = typename Act<ACT>::T;
    using M = ChunkGeom<ACT, DK, VT>;
    constexpr int C = M::C, NP = M::NP, NS = M::NS, PER = 16 / M::EB, MT = 64 * kMakers;
    constexpr int RP = DK / PER, NQ = C * RP / MT, RSTEP = MT / RP;     // q, k pieces of a row, of a maker's thread
    constexpr int VR = VT / PER, NV = C * VR / MT, VSTEP = MT / VR;     // v pieces
    constexpr int TT = C / 16, KK = C / 32, PAIRS = DK / 32;
    constexpr bool TWO = M::kDepth == 2;
    extern __shared__ __align__(16) unsigned char smem[];
    // by the chunk's parity where two chunks fit
    uint16_t *const Q0 = reinterpret_cast<uint16_t *>(smem), *const K0 = Q0 + M::kDepth * NP * M::QP,
             *const V0 = K0 + M::kDepth * NP * M::KP, *const Ps = V0 + M::kDepth * NP * M::VP;
    double *const G0 = reinterpret_cast<double *>(Ps + NS * M::PP);  // [2][C] by parity, as the next three
    float *const F0 = reinterpret_cast<float *>(G0 + 2 * C), *const E0 = F0 + 2 * C, *const factor = E0 + 2 * C;

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
    const int dk = a.s.dk, dv = a.s.dv, v0 = vt * VT, vcols = dv - v0 < VT ? dv - v0 : VT;
    int64_t len = a.L;
    if (a.lengths) len = a.lengths[b] < 0 ? 0 : a.lengths[b] < a.L ? a.lengths[b] : a.L;
    const int64_t begin = seg * p.seg_chunks * C, end = begin + p.seg_chunks * C < a.L ? begin + p.seg_chunks * C : a.L;
    const int64_t rows = len <= begin ? 0 : (len < end ? len : end) - begin;  // tokens of this segment
    const int chunks = (int)((rows + C - 1) / C);
    T *const y = static_cast<T *>(a.y) + (b * a.L + begin) * a.ld_y + h * dv + v0;

    if (wave >= M::kTakers) {
        // ---------------------------------------------------------------- makers
        // Ahead of the takers where both can issue: they have less to do, and wait on
        // memory (six rows of up to 1501 float32 tokens, 32 heads, with two passes: 134 us
        // against 152).
        __builtin_amdgcn_s_setprio(1);
        const int mt = tid - 64 * M::kTakers, maker = wave - M::kTakers;
        const T *const q = static_cast<const T *>(a.q) + (b * a.L + begin) * a.ld_q + h * a.s.qh / a.s.H * dk;
        const T *const k = static_cast<const T *>(a.k) + (b * a.L + begin) * a.ld_k + h * a.s.kh / a.s.H * dk;
        const T *const v = static_cast<const T *>(a.v) + (b * a.L + begin) * a.ld_v + h * a.s.vh / a.s.H * dv + v0;
        const float *const decay = a.decay ? a.decay + (a.ld_decay ? (b * a.L + begin) * a.ld_decay : 0) + h : nullptr;

        // The state-only form goes through its segment backwards, values weighted to the
        // segment's end: the full form starts where it ended, on tokens that may still be
        // in the Infinity Cache, and the state has no factor (65536 tokens, 16 heads: 2 to
        // 4 % of the call).
        auto first_token = [&](int c) { return (int64_t)(FULL ? c : chunks - 1 - c) * C; };

        // tokens of a chunk, on their way
        const int qr = mt / RP, qc = mt % RP * PER, vr = mt / VR, vc = mt % VR * PER;
        uint4 rq[NQ], rk[NQ], rv[NV];
        auto fetch = [&](int c) {
            const int64_t t0 = first_token(c), n = !FULL && t0 < 0 ? 0 : rows - t0;
            // rows past the last token read as zero by the bounds of the buffer
            const uint32_t last = n <= 0 ? 0 : (uint32_t)(n < C ? n - 1 : C - 1);
            const uint32_t sq = (uint32_t)a.ld_q * M::EB, sk = (uint32_t)a.ld_k * M::EB, sv = (uint32_t)a.ld_v * M::EB;
            const auto bq = make_region(q + t0 * a.ld_q, n <= 0 ? 0 : last * sq + dk * M::EB);
            const auto bk = make_region(k + t0 * a.ld_k, n <= 0 ? 0 : last * sk + dk * M::EB);
            const auto bv = make_region(v + t0 * a.ld_v, n <= 0 ? 0 : last * sv + vcols * M::EB);
            // of the thread's first pieces; the others' are formed here each time, not kept
            uint32_t oq = qc * M::EB + qr * sq, ok = qc * M::EB + qr * sk, ov = vc * M::EB + vr * sv;
            asm volatile("" : "+v"(oq), "+v"(ok), "+v"(ov));
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                if (FULL) rq[i] = load_piece<ACT, G, FULL>(bq, oq + i * RSTEP * sq, qc, dk);
                if constexpr (G < 8) __builtin_amdgcn_sched_barrier(0);  // elements are packed as they come
                rk[i] = load_piece<ACT, G, FULL>(bk, ok + i * RSTEP * sk, qc, dk);
                if constexpr (G < 8) __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rv[i] = load_piece<ACT, G, FULL>(bv, ov + i * VSTEP * sv, vc, vcols);
                if constexpr (G < 8) __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto store = [&](int c) {
            const int at = TWO ? c & 1 : 0;
            uint16_t *const Qs = Q0 + at * NP * M::QP, *const Ks = K0 + at * NP * M::KP, *const Vs = V0 + at * NP * M::VP;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                if (FULL) store_piece<ACT, M::QP>(Qs + (qr + i * RSTEP) * M::QS + qc, rq[i]);
                store_piece<ACT, M::KP>(Ks + (qr + i * RSTEP) * M::KS + qc, rk[i]);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) store_piece<ACT, M::VP>(Vs + (vr + i * VSTEP) * M::VS + vc, rv[i]);
        };

        // The last maker, which has the fewest tiles of P, forms a chunk's decays.
        // `error`: the state's factor as it should be over what float32 made of it,
        // handed on to the next chunk's factor, so that the factors' product over
        // many chunks is right to a rounding.
        float ra = 0.f;
        double total = 0.0, error = 1.0;
        auto fetch_decay = [&](int c) {
            const int64_t t0 = first_token(c), t = t0 + lane;
            ra = 0.f;
            if (decay && lane < C && (FULL || t0 >= 0) && t < rows) ra = bound_decay(decay[t * a.ld_decay]);
        };
        auto form_decays = [&](int c) {
            constexpr double kLog2e = 1.4426950408889634074;
            const int at = c & 1;
            const double g = scan_sum(ra * kLog2e);
            const double e = read_lane(g, C - 1);
            if constexpr (!FULL) {  // to the segment's end
                if (lane < C) E0[at * C + lane] = __builtin_amdgcn_exp2f((float)(total + (e - g)));
                total += e;
                return;
            }
            if (lane < C) {
                G0[at * C + lane] = g;
                F0[at * C + lane] = __builtin_amdgcn_exp2f((float)g);
                E0[at * C + lane] = __builtin_amdgcn_exp2f((float)(e - g));
            }
            const double f = exp2(e) * error;
            const float ff = (float)f;
            error = ff > 1e-30f ? 1.0 + (double)((float)(f - (double)ff) * __builtin_amdgcn_rcpf(ff)) : 1.0;
            if (lane == 0) factor[at] = ff;
        };

        // P[t][s] = exp(G_t - G_s) q_t . k_s for s <= t, in tiles (i, j) of 16 s x 16 t,
        // i <= j, N of them at once
        auto weigh_tiles = [&](int c, auto count, uint32_t tiles) {
            constexpr int N = decltype(count)::value;
            const int at = TWO ? c & 1 : 0;
            const uint16_t *kat[N], *qat[N];
            f32x4 x[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t code = tiles >> (4 * n) & 15;
                kat[n] = K0 + at * NP * M::KP + (16 * (code >> 2) + li) * M::KS + 8 * lg;
                qat[n] = Q0 + at * NP * M::QP + (16 * (code & 3) + li) * M::QS + 8 * lg;
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
            const double *const gs = G0 + (c & 1) * C;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t code = tiles >> (4 * n) & 15;
                const int t = 16 * (code & 3) + li, s = 16 * (code >> 2) + 4 * lg;
                uint16_t *const to = Ps + (t < 32 ? t * M::PS0 : 32 * M::PS0 + (t - 32) * M::PS1) + s;
                const double gt = gs[t];
                float o[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // the product may have overflowed with a later token's key, or one from before
                    // a reset, and is not used then: 0 times it would be NaN
                    const float f = __builtin_amdgcn_exp2f((float)(gt - gs[s + r]));
                    o[r] = s + r <= t && f != 0.f ? x[n][r] * f : 0.f;
                }
#pragma unroll
                for (int w = 0; w < NS; ++w) {
                    const uint32_t lo = take_part(o[0], o[1]);
                    *reinterpret_cast<uint2 *>(to + w * M::PP) = make_uint2(lo, take_part(o[2], o[3]));
                }
            }
        };
        auto weigh = [&](int c) {
            // codes 4 i + j of each maker's tiles
            constexpr uint32_t kTiles4[kMakers] = {0xb73, 0xa62, 0xf51, 0x0}, kTiles2[kMakers] = {0x1, 0x5, 0x0, 0x0};
            if (maker < 3)
                weigh_tiles(c, std::integral_constant<int, TT == 4 ? 3 : 1>{}, TT == 4 ? kTiles4[maker] : kTiles2[maker]);
            else if constexpr (TT == 4)
                weigh_tiles(c, std::integral_constant<int, 1>{}, kTiles4[3]);
        };

        // tiles above the diagonal that the products read: zero, once
        if (FULL)
            for (int i = mt; i < NS * M::PP; i += MT) Ps[i] = 0;
        if (chunks > 0) {
            fetch(0);
            if (maker == kMakers - 1) {
                fetch_decay(0);
                form_decays(0);
                fetch_decay(1);
            }
            store(0);
            fetch(1);
            __syncthreads();
            if (FULL) {
                weigh(0);
                __syncthreads();
            }
            for (int c = 0; c < chunks; ++c) {
                if (maker == kMakers - 1) {
                    form_decays(c + 1);
                    fetch_decay(c + 2);
                }
                if constexpr (!TWO) __syncthreads();
                if (c + 1 < chunks) store(c + 1);
                fetch(c + 2);
                __syncthreads();
                if (FULL) {
                    if (c + 1 < chunks) weigh(c + 1);
                    __syncthreads();
                }
            }
        }
        if (!FULL && vt == 0 && maker == kMakers - 1 && lane == 0) {
            const double f = exp2(total);
            reinterpret_cast<float2 *>(a.ws + p.off_decay)[bh * p.segs + seg] =
                make_float2((float)f, (float)(f - (double)(float)f));
        }
    } else {
        // ---------------------------------------------------------------- takers
        // the state: tile 2P + u, register r = key row 32 P + 8 lg + 4 u + r, value column li of the wave
        const int64_t cells = (int64_t)dk * dv;
        const int col = 16 * wave + li;
        // of the lane's first cell; rows 16 (t & ~1) + 4 (t & 1) + r further on.  The
        // compiler is kept from holding the cells' places from the first use to the last
        auto cell0 = [&](const float *x) {
            int g = lg;
            asm volatile("" : "+v"(g));
            return x + (int64_t)(8 * g) * dv + v0 + col;
        };
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
            for (int t = 0; t < 2 * PAIRS; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (from && col < vcols) {
                const float *at = cell0(from);
                const int left = dk - 8 * lg;
#pragma unroll
                for (int t = 0; t < 2 * PAIRS; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 16 * (t & ~1) + 4 * (t & 1) + r;
                        if (row < left) S[t][r] = at[row * dv];
                    }
            }
        }
        f32x4 acc[TT];
        uint4 va[KK][NP], vb[KK][3];
        // V of this wave's columns as an operand: value column li, tokens 32 kk + 8 lg + 0..7
        auto load_values = [&](int c) {
            const uint16_t *const Vs = V0 + (TWO ? c & 1 : 0) * NP * M::VP;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int w = 0; w < NP; ++w) {
                    const uint16_t *at = Vs + w * M::VP + (32 * kk + 8 * lg + (li >> 2)) * M::VS + 16 * wave + 4 * (li & 3);
                    const uint2 lo = read_transposed(at), hi = read_transposed(at + 4 * M::VS);
                    va[kk][w] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
        };
        // V weighted to the chunk's end, in parts
        auto weigh_values = [&](int c) {
            const float *const te = E0 + (c & 1) * C;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
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
                split8(x, vb[kk]);
            }
        };
        // acc = y / scale: exp(G_t) S^T q_t, then P V
        auto form_y = [&](int c) {
            const int buf = TWO ? c & 1 : 0;
            const uint16_t *const qat = Q0 + buf * NP * M::QP + li * M::QS + 8 * lg;
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
                if (pr == PAIRS - 1) load_values(c);
                __builtin_amdgcn_sched_barrier(0);
                float x[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) x[r] = S[2 * pr + r / 4][r % 4];
                uint4 sa[TT][NS];
                split8(x, sa[0]);
#pragma unroll
                for (int j = 1; j < TT; ++j)
#pragma unroll
                    for (int w = 0; w < NS; ++w) sa[j][w] = sa[0][w];
                mfma_tiles<TT>(sa, qb[pr & 1], acc);
            }
            const float *const fs = F0 + (c & 1) * C;
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                const float f = fs[16 * j + li];
                acc[j] = f != 0.f ? acc[j] * f : f32x4{0.f, 0.f, 0.f, 0.f};  // S^T q may have overflowed
            }
        };
        auto add_near = [&](int c) {
            const uint16_t *const pat0 = Ps + li * M::PS0 + 8 * lg, *const pat1 = Ps + 32 * M::PS0 + li * M::PS1 + 8 * lg;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                uint4 pb[TT][NS], vv[TT][NP];  // tiles j from 2 kk on
#pragma unroll
                for (int j = 2 * kk; j < TT; ++j) {
#pragma unroll
                    for (int w = 0; w < NS; ++w)
                        pb[j - 2 * kk][w] = *reinterpret_cast<const uint4 *>(
                            (j < 2 ? pat0 + 16 * j * M::PS0 : pat1 + 16 * (j - 2) * M::PS1 + 32 * kk) + w * M::PP);
#pragma unroll
                    for (int w = 0; w < NP; ++w) vv[j - 2 * kk][w] = va[kk][w];
                }
                if (kk == 0)
                    mfma_tiles<TT>(vv, pb, acc);
                else
                    mfma_tiles<2>(vv, pb, acc + 2 * kk);
            }
        };
        auto store_y = [&](int c) {
            const int64_t t0 = (int64_t)c * C, n = end - begin - t0;
            const int own = rows - t0 < C ? (int)(rows - t0) : C;  // tokens; rows past them are zero whatever the state
            const int vc = 16 * wave + 4 * lg;
            T *at = y + (t0 + li) * a.ld_y + vc;
            const bool whole = n >= C;
#pragma unroll
            for (int j = 0; j < TT; ++j, at += 16 * a.ld_y) {
                if (vc >= vcols || !(whole || 16 * j + li < n)) continue;
                const f32x4 o = 16 * j + li < own ? acc[j] * a.s.scale : f32x4{0.f, 0.f, 0.f, 0.f};
                if constexpr (G == 16 || (G == 8 && ACT == kBF16)) {
                    if constexpr (ACT == kBF16)
                        *reinterpret_cast<uint2 *>(at) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
                    else
                        *reinterpret_cast<float4 *>(at) = make_float4(o[0], o[1], o[2], o[3]);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (vc + r < vcols) Act<ACT>::st(at + r, o[r]);
                }
            }
        };
        auto advance = [&](int c) {
            const int buf = TWO ? c & 1 : 0;
            const uint16_t *const kat = K0 + buf * NP * M::KP + (8 * lg + (li >> 2)) * M::KS + 8 * (li & 3);
            // K transposed, KG tiles of key rows at a time, loaded one time ahead
            constexpr int KG = NP == 3 || DK == 32 || G != 16 ? 2 : 4, KPK = 2 * PAIRS / KG, KN = KK * KPK;
            uint4 ka[2][KG][NP];
            auto load = [&](int n) {
#pragma unroll
                for (int g = 0; g < KG; ++g) {
                    const int t = n % KPK * KG + g;
#pragma unroll
                    for (int w = 0; w < NP; ++w) {
                        const uint16_t *at = kat + w * M::KP + 32 * (n / KPK) * M::KS + 16 * (t & ~1) + 4 * (t & 1);
                        const uint2 lo = read_transposed(at), hi = read_transposed(at + 4 * M::KS);
                        ka[n & 1][g][w] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
            };
            load(0);
            if constexpr (FULL) {
                const float f = factor[c & 1];
#pragma unroll
                for (int t = 0; t < 2 * PAIRS; ++t) S[t] *= f;
            }
#pragma unroll
            for (int n = 0; n < KN; ++n) {
                const int kk = n / KPK, first = n % KPK * KG;
                if (n + 1 < KN) load(n + 1);
                uint4 vv[KG][3];
#pragma unroll
                for (int g = 0; g < KG; ++g)
#pragma unroll
                    for (int w = 0; w < 3; ++w) vv[g][w] = vb[kk][w];
                __builtin_amdgcn_sched_barrier(0);
                mfma_tiles<KG>(ka[n & 1], vv, S + first);
                __builtin_amdgcn_sched_barrier(0);
            }
        };

        if (chunks > 0) {
            __syncthreads();
            if (FULL) __syncthreads();
            for (int c = 0; c < chunks; ++c) {
                if constexpr (FULL) {
                    form_y(c);
                    weigh_values(c);
                    add_near(c);
                    if constexpr (TWO) __syncthreads();
                    advance(c);
                    store_y(c);
                } else {
                    load_values(c);
                    weigh_values(c);
                    advance(c);
                }
                __syncthreads();
                if constexpr (!TWO) {
                    __syncthreads();
                    if (FULL) __syncthreads();
                }
            }
        }
        float *const to = FULL ? a.state_out + bh * cells
                               : reinterpret_cast<float *>(a.ws) + (bh * p.segs + seg + 1) * cells;
        if ((!FULL || seg == p.segs - 1) && col < vcols) {
            float *at = const_cast<float *>(cell0(to));
            const int left = dk - 8 * lg;
#pragma unroll
            for (int t = 0; t < 2 * PAIRS; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * (t & ~1) + 4 * (t & 1) + r;
                    if (row < left) at[row * dv] = S[t][r];
                }
        }
    }
    if (FULL) {  // rows past the tokens
        const int col = tid % VT;
        if (col < vcols)
            for (int64_t t = (int64_t)chunks * C + tid / VT; t < end - begin; t += M::kThreads / VT)
                Act<ACT>::st(y + t * a.ld_y + col, 0.f);
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
    constexpr int AHEAD = 8;  // own states read before the first of them is overwritten
    for (int64_t s = 1; s < p.segs; s += AHEAD) {
        float own[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (s + j < p.segs) own[j] = slot[(s + j) * cells];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (s + j < p.segs) {
                const float2 f = factor[s + j - 1];
                x = fmaf(x, f.x, fmaf(x, f.y, own[j]));
                slot[(s + j) * cells] = x;
            }
    }
}

// ------------------------------------------------------------------ a few tokens

// Tokens of a prompt that the chunks are too long for.  Of eight shapes of 16 to 2048
// rows and heads, keys of 16 to 256: 10 bfloat16 tokens take all of them less time here
// (40 x 16 heads of 128 x 128: 31 us, 41 in chunks; 128 x 16 of 64 x 64: 39, 40), 12 not
// (43, 40).  A float32 chunk has six products for one: with 14 tokens shapes of many
// heads are faster here (38, 58), of few in chunks (1 x 16 heads: 13.4, 11.4), and with
// 16 most are (70, 58).
constexpr int short_prompt_tokens(int act) { return act == kF32 ? 14 : 10; }

// LDS of linattn_short_kernel: a token's q, k, decay, values, and y of four waves
constexpr int short_bytes(int tokens, int dk, int tile) {
    return tokens * (8 * dk + 8 + 4 * tile + 4 * tile * (kThreads / kWave));
}

// A prompt of at most so many tokens, all float32: the layout of one token's kernel
// (LANES threads of V value columns a key row), the state read once, taken through
// the tokens in registers and written once.  Bound by the state's way out, and past
// some 8 tokens by the vector ALUs.  (Going on from a state, 37 x 4 heads of 256 x 256,
// 4 float32 tokens: 18.9 us, 61.4 in chunks; 44 x 24 of 16 x 16, 8 bfloat16 ones: 14.9,
// 20.3 in chunks.)
template <int ACT, int LANES, int V, bool DECAY>
__global__ __launch_bounds__(kThreads) void linattn_short_kernel(LinAttnArgs a, int vtiles) {
    using T = typename Act<ACT>::T;
    typedef float vec __attribute__((ext_vector_type(V)));
    constexpr int ROWS = kThreads / LANES, TILE = LANES * V, FLY = LANES == 8 ? 8 : 16;
    extern __shared__ __align__(16) unsigned char smem[];
    const int64_t unit = blockIdx.x / vtiles, b = unit / a.s.H, h = unit - b * a.s.H;
    const int tid = threadIdx.x, lane = tid % LANES, row0 = tid / LANES, dk = a.s.dk, dv = a.s.dv;
    const int L = (int)a.L, col0 = (int)(blockIdx.x - unit * vtiles) * TILE, col = col0 + lane * V;
    int len = L;
    if (a.lengths) len = a.lengths[b] < 0 ? 0 : a.lengths[b] < L ? a.lengths[b] : L;
    vec *const part = reinterpret_cast<vec *>(smem);                    // [waves][L][LANES]
    float *const vs = reinterpret_cast<float *>(part + kThreads / kWave * L * LANES);  // [L][TILE]
    float2 *const qk = reinterpret_cast<float2 *>(vs + L * TILE);       // [L][dk]: q scale, k
    float2 *const g = qk + L * dk;                                      // [L]
    const T *const q = static_cast<const T *>(a.q) + b * L * a.ld_q + h * a.s.qh / a.s.H * dk;
    const T *const k = static_cast<const T *>(a.k) + b * L * a.ld_k + h * a.s.kh / a.s.H * dk;
    const T *const v = static_cast<const T *>(a.v) + b * L * a.ld_v + h * a.s.vh / a.s.H * dv + col0;
    for (int i = tid; i < len * dk; i += kThreads) {
        const int t = i / dk, c = i - t * dk;
        qk[i] = make_float2(a.s.scale * Act<ACT>::ld(q + t * a.ld_q + c), Act<ACT>::ld(k + t * a.ld_k + c));
    }
    for (int i = tid; i < len * TILE; i += kThreads) {
        const int t = i / TILE, c = i % TILE;
        vs[i] = col0 + c < dv ? Act<ACT>::ld(v + t * a.ld_v + c) : 0.f;
    }
    if (tid < len)
        g[tid] = DECAY ? decay_factor(a.decay[a.ld_decay ? (b * L + tid) * a.ld_decay + h : h]) : float2{};
    __syncthreads();
    const int64_t base = unit * (int64_t)dk * dv + col;
    const bool own = col < dv;  // V divides dv
    const int wave = tid / kWave;
    for (int n0 = 0; n0 * ROWS < dk; n0 += FLY) {
        vec s[FLY];
#pragma unroll
        for (int n = 0; n < FLY; ++n) {
            const int i = row0 + (n0 + n) * ROWS;
            s[n] = vec{};
            if (a.state_in && own && i < dk) s[n] = *reinterpret_cast<const vec *>(a.state_in + base + (int64_t)i * dv);
        }
        for (int t = 0; t < len; ++t) {
            const vec x = reinterpret_cast<const vec *>(vs + t * TILE)[lane];
            const float2 f = g[t];
            vec y = {};
#pragma unroll
            for (int n = 0; n < FLY; ++n) {
                const int i = row0 + (n0 + n) * ROWS;
                if (i < dk) {
                    const float2 w = qk[t * dk + i];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        s[n][e] = decayed<DECAY>(f, s[n][e], w.y * x[e]);
                        y[e] = fmaf(w.x, s[n][e], y[e]);
                    }
                }
            }
#pragma unroll
            for (int m = LANES; m < kWave; m <<= 1)
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] += __shfl_xor(y[e], m);
            if ((tid & (kWave - 1)) < LANES) {
                vec *const at = part + (wave * L + t) * LANES + lane;
                *at = n0 == 0 ? y : *at + y;
            }
        }
#pragma unroll
        for (int n = 0; n < FLY; ++n) {
            const int i = row0 + (n0 + n) * ROWS;
            if (own && i < dk) *reinterpret_cast<vec *>(a.state_out + base + (int64_t)i * dv) = s[n];
        }
    }
    __syncthreads();
    T *const y = static_cast<T *>(a.y) + b * L * a.ld_y + h * dv + col0;
    const float *const sums = reinterpret_cast<const float *>(part);
    for (int i = tid; i < L * TILE; i += kThreads) {
        const int t = i / TILE, c = i % TILE;
        if (col0 + c >= dv) continue;
        float o = 0.f;
        if (t < len) o = (sums[i] + sums[L * TILE + i]) + (sums[2 * L * TILE + i] + sums[3 * L * TILE + i]);
        Act<ACT>::st(y + t * a.ld_y + c, o);
    }
}

// ------------------------------------------------------------------ one token

// One workgroup for a batch row, a head and a tile of LANES * V value columns:
// LANES threads of V columns a key row, 256 / LANES rows at a time, every row's
// load of a thread in flight before the first is used (in turns of 16).
// Bound by the state's way in and out.
template <int ACT, int LANES, int V, bool DECAY>
__global__ __launch_bounds__(kThreads) void linattn_token_kernel(LinAttnArgs a, int vtiles) {
    using T = typename Act<ACT>::T;
    typedef float vec __attribute__((ext_vector_type(V)));
    constexpr int ROWS = kThreads / LANES, TILE = LANES * V, FLY = LANES == 8 ? 8 : 16;
    __shared__ float2 qk[kMaxDk];  // q scale, k
    __shared__ vec part[kThreads / kWave][LANES];
    const int64_t unit = blockIdx.x / vtiles, b = unit / a.s.H, h = unit - b * a.s.H;
    const int tid = threadIdx.x, lane = tid % LANES, row0 = tid / LANES, dk = a.s.dk, dv = a.s.dv;
    const int col = (int)(blockIdx.x - unit * vtiles) * TILE + lane * V;
    int64_t src = b;
    if (a.src_rows) {
        const int s = a.src_rows[b];
        if (s >= 0 && s < a.s.B) src = s;
    }
    const float *in = a.state_in + (src * a.s.H + h) * (int64_t)dk * dv + col;
    float *out = a.state_out + unit * (int64_t)dk * dv + col;
    const bool own = col < dv;  // V divides dv
    vec s[FLY];
#pragma unroll
    for (int n = 0; n < FLY; ++n) {
        const int i = row0 + n * ROWS;
        if (own && i < dk) s[n] = __builtin_nontemporal_load(reinterpret_cast<const vec *>(in + (int64_t)i * dv));
    }
    for (int i = tid; i < dk; i += kThreads)
        qk[i] = make_float2(
            a.s.scale * Act<ACT>::ld(static_cast<const T *>(a.q) + b * a.ld_q + h * a.s.qh / a.s.H * dk + i),
            Act<ACT>::ld(static_cast<const T *>(a.k) + b * a.ld_k + h * a.s.kh / a.s.H * dk + i));
    const float2 g = DECAY ? decay_factor(a.decay[a.ld_decay ? b * a.ld_decay + h : h]) : float2{};
    vec v = {}, y = {};
    if (own) {
        const T *at = static_cast<const T *>(a.v) + b * a.ld_v + h * a.s.vh / a.s.H * dv + col;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = Act<ACT>::ld(at + e);
    }
    __syncthreads();
    for (int n0 = 0; n0 * ROWS < dk; n0 += FLY) {
        if (n0 > 0)
#pragma unroll
            for (int n = 0; n < FLY; ++n) {
                const int i = row0 + (n0 + n) * ROWS;
                if (own && i < dk) s[n] = __builtin_nontemporal_load(reinterpret_cast<const vec *>(in + (int64_t)i * dv));
            }
#pragma unroll
        for (int n = 0; n < FLY; ++n) {
            const int i = row0 + (n0 + n) * ROWS;
            if (own && i < dk) {
                const float2 w = qk[i];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    s[n][e] = decayed<DECAY>(g, s[n][e], w.y * v[e]);
                    y[e] = fmaf(w.x, s[n][e], y[e]);
                }
                __builtin_nontemporal_store(s[n], reinterpret_cast<vec *>(out + (int64_t)i * dv));
            }
        }
    }
    // the rows' parts of y: within a wave, then over the waves
#pragma unroll
    for (int m = LANES; m < kWave; m <<= 1)
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] += __shfl_xor(y[e], m);
    if ((tid & (kWave - 1)) < LANES) part[tid / kWave][lane] = y;
    __syncthreads();
    if (tid < LANES && own) {
        const vec o = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
        T *at = static_cast<T *>(a.y) + b * a.ld_y + h * dv + col;
#pragma unroll
        for (int e = 0; e < V; ++e) Act<ACT>::st(at + e, o[e]);
    }
}

// One token (short_prompt false) or a short prompt.
template <int ACT, int LANES, int V, bool DECAY>
hipError_t launch_token(const LinAttnArgs &a, bool short_prompt, hipStream_t stream) {
    const int vtiles = (a.s.dv + LANES * V - 1) / (LANES * V);
    const dim3 grid((unsigned)(a.s.B * a.s.H * vtiles));
    if (!short_prompt) {
        linattn_token_kernel<ACT, LANES, V, DECAY><<<grid, kThreads, 0, stream>>>(a, vtiles);
        return hipGetLastError();
    }
    const int bytes = short_bytes((int)a.L, a.s.dk, LANES * V);
    const auto kernel = linattn_short_kernel<ACT, LANES, V, DECAY>;
    if (bytes > 65536) {
        const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (err != hipSuccess) return err;
    }
    kernel<<<grid, kThreads, bytes, stream>>>(a, vtiles);
    return hipGetLastError();
}

template <int ACT, int LANES, int V>
hipError_t launch_token(const LinAttnArgs &a, bool short_prompt, hipStream_t stream) {
    return a.decay ? launch_token<ACT, LANES, V, true>(a, short_prompt, stream)
                   : launch_token<ACT, LANES, V, false>(a, short_prompt, stream);
}

// 16-byte pieces of the state where its rows allow them.  128 value columns a
// workgroup where that gives two a CU, else 32 (batch 1, 16 heads of 128 x 128:
// 4.6 us, 11.5 with whole heads).
template <int ACT>
hipError_t launch_token(const LinAttnArgs &a, bool short_prompt, hipStream_t stream) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.state_in) | reinterpret_cast<uintptr_t>(a.state_out);
    if (bits % 16 != 0 || a.s.dv % 4 != 0) return launch_token<ACT, 64, 1>(a, short_prompt, stream);
    const int64_t units = a.s.B * a.s.H;
    if (units * ((a.s.dv + 127) / 128) >= 512) return launch_token<ACT, 32, 4>(a, short_prompt, stream);
    return launch_token<ACT, 8, 4>(a, short_prompt, stream);
}

// Padded key width, and the granule of 16, 8 bytes or an element that all rows allow.
int padded_dk(int dk) { return dk <= 32 ? 32 : dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }

LinAttnPlan linattn_plan(const LinAttnShape &s, int64_t L) {
    LinAttnPlan p;
    p.chunk = s.act == kBF16 && s.dk <= 128 ? 64 : 32;
    // Value columns of a workgroup and segments of the prompt: the least of rounds of
    // workgroups x chunks of one.
    //   One workgroup a CU; two of 64 columns and up to 32 bfloat16 keys, which leave room
    //     (8 rows of 2000 tokens, 16 heads of 32 x 32: 46 us against 59).
    //   64 columns take kNarrow of the time of 128 a chunk (77 tokens of 16 heads: 14.3 us
    //     against 16.4; of 17 shapes of both types, key widths of 32 to 256, this picks the
    //     faster tile or one within 5 % at all but 8 x 700 tokens, 32 heads of 32 x 128:
    //     44.6 us, 38 with 128 columns).  128 are for more than 64 where the LDS holds two chunks of them
    //     and the registers of three waves a SIMD the state.
    //   Segments cost a second pass over k and v, kAgain of the full one (0.4 takes the same
    //     time at the 17 shapes).  (Cutting rows of
    //     their own lengths finer, for balance, did not pay: six rows of up to 1501 float32
    //     tokens, 32 heads: 152 us in four segments, 124 us whole.)
    constexpr double kNarrow = 0.75, kAgain = 0.6;
    constexpr int64_t kCUs = 256, kFew = 4;  // kFew: chunks of a segment, at least
    const int64_t chunks = (L + p.chunk - 1) / p.chunk;
    int64_t segs = 1;
    double best = -1.0;
    for (int vt : {64, 128}) {
        if (vt == 128 && (s.dv <= 64 || s.dk > (s.act == kBF16 ? 128 : 64))) continue;
        const int vtiles = (s.dv + vt - 1) / vt;
        const int64_t groups = s.B * s.H * vtiles, kSlots = vt == 64 && s.dk <= 32 && s.act == kBF16 ? 2 * kCUs : kCUs;
        for (int64_t n = 1; n == 1 || (n * kFew <= chunks && groups * n < 2 * kSlots); ++n) {
            const double cost = (double)((groups * n + kSlots - 1) / kSlots * ((chunks + n - 1) / n)) *
                                (n > 1 ? 1 + kAgain : 1) * (vt == 64 ? kNarrow : 1);
            if (best < 0 || cost < best) {
                best = cost;
                segs = n;
                p.vt = vt;
                p.vtiles = vtiles;
            }
        }
    }
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
    return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : e;
}

template <int ACT, int DK, int VT, int G, bool FULL>
hipError_t launch_chunks(const LinAttnArgs &a, const LinAttnPlan &p, hipStream_t stream) {
    using M = ChunkGeom<ACT, DK, VT>;
    const auto kernel = linattn_chunk_kernel<ACT, DK, VT, G, FULL>;
    if (M::kBytes > 65536) {
        const hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, M::kBytes);
        if (err != hipSuccess) return err;
    }
    const int64_t units = a.s.B * a.s.H * p.segs;
    kernel<<<dim3((unsigned)((units + 7) / 8 * 8 * p.vtiles)), M::kThreads, M::kBytes, stream>>>(a, p);
    return hipGetLastError();
}

template <int ACT, int DK, int VT, int G>
hipError_t launch_prompt(const LinAttnArgs &a, const LinAttnPlan &p, hipStream_t stream) {
    if (p.segs > 1) {
        hipError_t err = launch_chunks<ACT, DK, VT, G, false>(a, p, stream);
        if (err != hipSuccess) return err;
        const dim3 grid((unsigned)(a.s.B * a.s.H), (unsigned)((a.s.dk * a.s.dv + kThreads - 1) / kThreads));
        linattn_join_kernel<<<grid, kThreads, 0, stream>>>(a, p);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    return launch_chunks<ACT, DK, VT, G, true>(a, p, stream);
}

template <int ACT, int DK, int G>
hipError_t launch_prompt(const LinAttnArgs &a, const LinAttnPlan &p, hipStream_t stream) {
    // (element loads take more registers than a workgroup of 128 columns has)
    if constexpr (DK <= (ACT == kBF16 ? 128 : 64) && G >= 8)
        if (p.vt == 128) return launch_prompt<ACT, DK, 128, G>(a, p, stream);
    LinAttnPlan narrow = p;
    narrow.vt = 64;
    narrow.vtiles = (a.s.dv + 63) / 64;
    return launch_prompt<ACT, DK, 64, G>(a, narrow, stream);
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
    if (a.L > 0 && a.L <= short_prompt_tokens(a.s.act))
        return a.s.act == kBF16 ? launch_token<kBF16>(a, true, stream) : launch_token<kF32>(a, true, stream);
    const LinAttnPlan p = linattn_plan(a.s, a.L);
    return a.s.act == kBF16 ? launch_prompt<kBF16>(a, p, stream) : launch_prompt<kF32>(a, p, stream);
}

hipError_t launch_linattn_decode(const LinAttnArgs &a, hipStream_t stream) {
    return a.s.act == kBF16 ? launch_token<kBF16>(a, false, stream) : launch_token<kF32>(a, false, stream);
}

}  // namespace hm
