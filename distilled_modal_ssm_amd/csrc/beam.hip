// beam.hip -- beam search: the best continuations of every group of beams, and
// the move of the layers' states to where their beams went.
//
// score(k, v) = scores[k] + x_kv - max_k - log sum_v exp(x_kv - max_k), the best
// `select` of beams x vocab, equal ones in the order of k * vocab + v.
//
// A beam's scores order as its logits, so the rows are cut into segments of
// which each hands on its best `select` logits with the segment's maximum and
// sum of exponentials (one pass over the logits); a second kernel, one workgroup
// a group, joins the segments' statistics and takes the best of what they
// handed on.  Both find their best through the same block_best below.
#include "hm_internal.hpp"

namespace hm {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kMaxSelect = 64;
constexpr int kList = 1024;          // continuations that pass block_best's bound, at most
constexpr int kNone = 0x7fffffff;    // index of "no continuation"

constexpr float kNever = -__builtin_inff();

struct Best {
    float x;
    int32_t i;
};

__device__ __forceinline__ bool before(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
    return x;
}

// The 64 lanes' values in decreasing order.
__device__ __forceinline__ float wave_sort(float x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const float y = __shfl_xor(x, j);
            const bool up = (lane & k) != 0, low = (lane & j) == 0;
            x = (low != up) ? fmaxf(x, y) : fminf(x, y);
        }
    return x;
}

__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x);
}

struct BestShared {
    Best list[kList];
    float bound[kWaves];
    Best lead[kWaves];
    int count;
};

// The best n (<= 64) of the workgroup's values, kThreads x E in registers, by
// (value, lowest index), into out[0 .. n) in that order; values of -infinity are
// absent, and missing places get {-infinity, kNone}.  Indices differ.
//
// The n-th largest of a wave's 64 lane maxima bounds the n-th best value from
// below, and so does the largest of the waves' bounds: what is below it is out.
// The rest, n and a few more, is listed and each entry put at its rank.  Values
// that are equal many times over can overrun the list; then the best are taken
// out one by one instead.
template <int E>
__device__ __forceinline__ void block_best(const float (&x)[E], const int (&idx)[E], int n, BestShared &sh, Best *out) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float top = kNever;
#pragma unroll
    for (int e = 0; e < E; ++e) top = fmaxf(top, x[e]);
    const float sorted = wave_sort(top);
    const float nth = __shfl(sorted, n - 1);
    if (lane == 0) sh.bound[wave] = nth;
    if (tid == 0) sh.count = 0;
    for (int i = tid; i < n; i += kThreads) out[i] = {kNever, kNone};
    __syncthreads();
    float bound = sh.bound[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) bound = fmaxf(bound, sh.bound[w]);
    if (top >= bound && top > kNever) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (x[e] >= bound && x[e] > kNever) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kList) sh.list[at] = {x[e], idx[e]};
            }
    }
    __syncthreads();
    const int count = sh.count;
    if (count <= kList) {
        for (int i = tid; i < count; i += kThreads) {
            const Best me = sh.list[i];
            int rank = 0;
            for (int j = 0; j < count; ++j) rank += before(sh.list[j].x, sh.list[j].i, me.x, me.i);
            if (rank < n) out[rank] = me;
        }
    } else {
        float lx = __builtin_inff();
        int li = -1;  // the last one taken
        for (int r = 0; r < n; ++r) {
            float bx = kNever;
            int bi = kNone;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (before(lx, li, x[e], idx[e]) && x[e] > kNever && before(x[e], idx[e], bx, bi)) {
                    bx = x[e];
                    bi = idx[e];
                }
#pragma unroll
            for (int m = 32; m > 0; m >>= 1) {
                const float ox = __shfl_xor(bx, m);
                const int oi = __shfl_xor(bi, m);
                if (before(ox, oi, bx, bi)) {
                    bx = ox;
                    bi = oi;
                }
            }
            if (lane == 0) sh.lead[wave] = {bx, bi};
            __syncthreads();
            lx = sh.lead[0].x;
            li = sh.lead[0].i;
            for (int w = 1; w < kWaves; ++w)
                if (before(sh.lead[w].x, sh.lead[w].i, lx, li)) {
                    lx = sh.lead[w].x;
                    li = sh.lead[w].i;
                }
            if (tid == 0) out[r] = {lx, li};
            __syncthreads();
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------------ segments

constexpr int kSegE = 32;                       // logits of a thread
constexpr int kSegment = kThreads * kSegE;

struct SelectPlan {
    int64_t segs;
    size_t off_stat, off_best, bytes;  // float2 [rows][segs] (max, sum); Best [rows][segs][select]
};

SelectPlan select_plan(int64_t groups, int64_t beams, int64_t vocab, int64_t select) {
    SelectPlan p;
    p.segs = (vocab + kSegment - 1) / kSegment;
    p.off_stat = 0;
    p.off_best = ((size_t)(groups * beams * p.segs) * sizeof(float2) + 255) / 256 * 256;
    p.bytes = p.off_best + (size_t)(groups * beams * p.segs * select) * sizeof(Best);
    return p;
}

template <int ACT>
__global__ __launch_bounds__(kThreads) void beam_segment_kernel(BeamSelectArgs a, SelectPlan p) {
    using T = typename Act<ACT>::T;
    __shared__ BestShared sh;
    __shared__ Best best[kMaxSelect];
    __shared__ float red[kWaves];
    const int64_t row = blockIdx.x / p.segs, seg = blockIdx.x - row * p.segs;
    const int tid = threadIdx.x, n = (int)a.select;
    // a beam that has ended or is not alive has no continuation of its own here
    if (a.scores[row] == kNever || (a.finished && a.finished[row])) return;
    const T *x = static_cast<const T *>(a.logits) + row * a.ld;
    float val[kSegE];
    int idx[kSegE];
    float top = kNever;
#pragma unroll
    for (int e = 0; e < kSegE; ++e) {
        idx[e] = (int)(seg * kSegment) + e * kThreads + tid;
        const float f = idx[e] < a.vocab ? Act<ACT>::ld(x + idx[e]) : kNever;
        val[e] = f == f ? f : kNever;
        top = fmaxf(top, val[e]);
    }
    top = wave_max(top);
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, red[w]);
    __syncthreads();
    float sum = 0.f;
    if (top > kNever) {
#pragma unroll
        for (int e = 0; e < kSegE; ++e) sum += val[e] == top ? 1.f : __expf(val[e] - top);
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
    if ((tid & 63) == 0) red[tid >> 6] = sum;
    block_best<kSegE>(val, idx, n, sh, best);
    const int64_t at = row * p.segs + seg;
    if (tid == 0)
        reinterpret_cast<float2 *>(a.ws + p.off_stat)[at] = make_float2(top, (red[0] + red[1]) + (red[2] + red[3]));
    if (tid < n) reinterpret_cast<Best *>(a.ws + p.off_best)[at * n + tid] = best[tid];
}

// ------------------------------------------------------------------ groups

constexpr int kPickE = 8;

__global__ __launch_bounds__(kThreads) void beam_pick_kernel(BeamSelectArgs a, SelectPlan p) {
    __shared__ BestShared sh;
    __shared__ Best best[kMaxSelect];
    __shared__ float score0[kMaxSelect], top[kMaxSelect], lse[kMaxSelect];  // lse: log of the sum, after the maximum
    __shared__ bool ended[kMaxSelect];
    const int64_t g = blockIdx.x;
    const int tid = threadIdx.x, K = (int)a.beams, n = (int)a.select, V = (int)a.vocab;
    const float2 *stat = reinterpret_cast<const float2 *>(a.ws + p.off_stat) + g * K * p.segs;
    const Best *cand = reinterpret_cast<const Best *>(a.ws + p.off_best) + g * K * p.segs * n;
    if (tid < K) {
        const float s = a.scores[g * K + tid];
        const bool f = a.finished && a.finished[g * K + tid];
        float m = kNever, sum = 0.f;
        if (!f && s > kNever) {
            for (int64_t i = 0; i < p.segs; ++i) m = fmaxf(m, stat[tid * p.segs + i].x);
            for (int64_t i = 0; i < p.segs; ++i) {
                const float2 st = stat[tid * p.segs + i];
                if (st.x > kNever) sum += st.x == m ? st.y : st.y * expf(st.x - m);
            }
        }
        score0[tid] = s;
        ended[tid] = f;
        top[tid] = m;
        lse[tid] = logf(sum);
    }
    if (tid < kMaxSelect) best[tid] = {kNever, kNone};
    __syncthreads();
    const int64_t per = p.segs * n, total = K * per;
    float val[kPickE + 1];
    int idx[kPickE + 1];
    for (int64_t c0 = 0; c0 < total; c0 += kThreads * kPickE) {
#pragma unroll
        for (int e = 0; e < kPickE; ++e) {
            const int64_t c = c0 + e * kThreads + tid;
            val[e] = kNever;
            idx[e] = kNone;
            if (c < total) {
                const int k = (int)(c / per);
                if (ended[k]) {  // one continuation, in the place of the beam's first
                    if (c == k * per) {
                        val[e] = score0[k];
                        idx[e] = k * V + (int)a.end_token;
                    }
                } else if (score0[k] > kNever) {
                    const Best x = cand[c];
                    if (x.i != kNone) {
                        const float d = x.x == top[k] ? 0.f : x.x - top[k];
                        val[e] = score0[k] + (d - lse[k]);
                        idx[e] = k * V + x.i;
                    }
                }
            }
        }
        // the best so far stay in
        val[kPickE] = tid < n ? best[tid].x : kNever;
        idx[kPickE] = tid < n ? best[tid].i : kNone;
        __syncthreads();
        block_best<kPickE + 1>(val, idx, n, sh, best);
    }
    // fewer than n continuations: the first others, all of score -infinity
    if (tid == 0 && best[n - 1].i == kNone) {
        int have = 0;
        while (have < n && best[have].i != kNone) ++have;
        const int found = have;
        for (int f = 0; have < n; ++f) {
            bool taken = false;
            for (int j = 0; j < found; ++j) taken |= best[j].i == f;
            if (!taken) best[have++].i = f;
        }
    }
    __syncthreads();
    if (tid < n) {
        const int parent = best[tid].i / V, token = best[tid].i - parent * V;
        a.out_scores[g * n + tid] = best[tid].x;
        a.out_tokens[g * n + tid] = token;
        a.out_parents[g * n + tid] = parent;
        if (a.out_finished) a.out_finished[g * n + tid] = ended[parent] || token == a.end_token;
    }
}

// ------------------------------------------------------------------ reorder

constexpr int kBuffers = 96;  // buffers of a launch
struct ReorderArgs {
    const int32_t *parents;
    int beams, n;
    int first[kBuffers + 1];      // first workgroup of each buffer, in each group
    unsigned char *buf[kBuffers];
    int64_t bytes[kBuffers];
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kMoves = 4;  // pieces of a row that a thread moves, one after the other

// One workgroup for a group, a buffer and kMoves * 256 pieces of its rows.  A
// thread moves its piece in every row of the group, all reads before the first
// write, so the rows need no other order and no second buffer.  A parent is read
// once however many beams continue it; a row that stays is not touched, but as
// some other's parent.
template <typename T, int K>
__global__ __launch_bounds__(kThreads) void beam_reorder_kernel(ReorderArgs a) {
    __shared__ uint64_t kids[kMaxSelect];  // beams, but itself, that continue each beam
    const int tid = threadIdx.x;
    const int32_t *parent = a.parents + (int64_t)blockIdx.y * a.beams;
    if (tid < a.beams) {
        uint64_t m = 0;
        for (int k = 0; k < a.beams; ++k)
            if (k != tid && parent[k] == tid) m |= uint64_t(1) << k;
        kids[tid] = m;
    }
    int i = 0;
    while (i + 1 < a.n && (int)blockIdx.x >= a.first[i + 1]) ++i;
    const int64_t pieces = a.bytes[i] / (int64_t)sizeof(T);
    const int64_t first = ((int64_t)blockIdx.x - a.first[i]) * (kMoves * kThreads) + tid;
    T *rows = reinterpret_cast<T *>(a.buf[i]) + (int64_t)blockIdx.y * a.beams * pieces;
    __syncthreads();
    for (int64_t at = first; at < pieces && at < first + kMoves * kThreads; at += kThreads) {
        T x[K];
#pragma unroll
        for (int p = 0; p < K; ++p)
            if (p < a.beams && uniform(kids[p]) != 0) x[p] = rows[p * pieces + at];
#pragma unroll
        for (int p = 0; p < K; ++p) {
            for (uint64_t m = p < a.beams ? uniform(kids[p]) : 0; m != 0; m &= m - 1)
                rows[__builtin_ctzll(m) * pieces + at] = x[p];
        }
    }
}

template <typename T>
void launch_reorder(const ReorderArgs &a, int64_t groups, hipStream_t stream) {
    const dim3 grid((unsigned)a.first[a.n], (unsigned)groups);
    // registers for a piece of every beam
    if (a.beams <= 8)
        beam_reorder_kernel<T, 8><<<grid, kThreads, 0, stream>>>(a);
    else if (a.beams <= 16)
        beam_reorder_kernel<T, 16><<<grid, kThreads, 0, stream>>>(a);
    else
        beam_reorder_kernel<T, 64><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

size_t beam_select_workspace(int64_t groups, int64_t beams, int64_t vocab, int64_t select) {
    return select_plan(groups, beams, vocab, select).bytes;
}

hipError_t launch_beam_select(const BeamSelectArgs &a, hipStream_t stream) {
    const SelectPlan p = select_plan(a.groups, a.beams, a.vocab, a.select);
    const dim3 grid((unsigned)(a.groups * a.beams * p.segs));
    if (a.act == kBF16)
        beam_segment_kernel<kBF16><<<grid, kThreads, 0, stream>>>(a, p);
    else
        beam_segment_kernel<kF32><<<grid, kThreads, 0, stream>>>(a, p);
    beam_pick_kernel<<<dim3((unsigned)a.groups), kThreads, 0, stream>>>(a, p);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(int64_t groups, int64_t beams, const int32_t *parents, int64_t n, void *const *buffers,
                               const int64_t *row_bytes, hipStream_t stream) {
    if (beams == 1) return hipSuccess;
    // buffers of one piece size share a launch: 16 bytes where all rows allow it (8
    // for more than 16 beams: a thread holds a piece of each), else 4, else 1
    const int widest = beams <= 16 ? 16 : 8;
    for (int size : {widest, 4, 1}) {
        ReorderArgs a;
        a.parents = parents;
        a.beams = (int)beams;
        a.n = 0;
        a.first[0] = 0;
        for (int64_t i = 0; i <= n; ++i) {
            if (i < n && row_bytes[i] > 0) {
                const uintptr_t bits = reinterpret_cast<uintptr_t>(buffers[i]) | (uintptr_t)row_bytes[i];
                const int fits = bits % widest == 0 ? widest : bits % 4 == 0 ? 4 : 1;
                if (fits == size) {
                    const int64_t block = (int64_t)size * kMoves * kThreads;
                    a.buf[a.n] = static_cast<unsigned char *>(buffers[i]);
                    a.bytes[a.n] = row_bytes[i];
                    a.first[a.n + 1] = a.first[a.n] + (int)((row_bytes[i] + block - 1) / block);
                    ++a.n;
                }
            }
            // (a buffer has at most 2^26 workgroups)
            if (a.n == kBuffers || a.first[a.n] >= 1 << 29 || (i == n && a.n > 0)) {
                if (size == 16) launch_reorder<u32x4>(a, groups, stream);
                if (size == 8) launch_reorder<u32x2>(a, groups, stream);
                if (size == 4) launch_reorder<uint32_t>(a, groups, stream);
                if (size == 1) launch_reorder<uint8_t>(a, groups, stream);
                const hipError_t err = hipGetLastError();
                if (err != hipSuccess) return err;
                a.n = 0;
            }
        }
    }
    return hipSuccess;
}

}  // namespace hm
