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
//
// What bounds it (MI355X): a segment's fixed steps (the lane sort, the listing, the
// ranks) and its exponentials, some 24 vector instructions a logit, of which 7 are
// the softmax's; 32 x 8 rows of 131072 float32 logits take 42 us of segments (3.2
// TB/s) and 12 us of picks.  Segments of 2048 logits took 110 us in all, of 4096 83,
// of 8192 59, of 16384 58.  Small calls: two launches and the calling program.
//
// The reorder is bound by memory (64 beams over 24 layers: 1.49 GB in 320 us, 4.7
// TB/s); each thread moves one piece of every row of its group.
#include "hm_internal.hpp"

namespace hm {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kMaxSelect = 64;
constexpr int kList = 1024;          // continuations that pass block_best's bound, at most
constexpr int kNone = 0x7fffffff;    // index of "no continuation"

constexpr float kNever = -__builtin_inff(), kLowest = -3.402823466e38f;

struct Best {
    float x;
    int32_t i;
};

__device__ __forceinline__ bool before(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

// x of the lane whose number differs in bit J.
template <int J>
__device__ __forceinline__ float across(float x) {
    const int b = __float_as_int(x);
    if constexpr (J == 1) return __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0xb1, 0xf, 0xf, false));  // quad 1 0 3 2
    if constexpr (J == 2) return __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x4e, 0xf, 0xf, false));  // quad 2 3 0 1
    if constexpr (J == 4) {  // banks 0 and 2 of a row from 4 lanes on, 1 and 3 from 4 lanes before
        const int up = __builtin_amdgcn_update_dpp(0, b, 0x104, 0xf, 0x5, false);
        return __int_as_float(__builtin_amdgcn_update_dpp(up, b, 0x114, 0xf, 0xa, false));
    }
    if constexpr (J == 8) return __int_as_float(__builtin_amdgcn_update_dpp(0, b, 0x128, 0xf, 0xf, false));  // row turned by 8
    return __shfl_xor(x, J);
}

template <int K, int J>
__device__ __forceinline__ void sort_steps(float &x, int lane) {
    const float y = across<J>(x);
    const bool large = ((lane & J) == 0) == ((lane & K) == 0);
    x = large ? fmaxf(x, y) : fminf(x, y);
    if constexpr (J > 1) sort_steps<K, J / 2>(x, lane);
}

// The 64 lanes' values in decreasing order (a bitonic network).
__device__ __forceinline__ float wave_sort(float x) {
    const int lane = threadIdx.x & 63;
    sort_steps<2, 1>(x, lane);
    sort_steps<4, 2>(x, lane);
    sort_steps<8, 4>(x, lane);
    sort_steps<16, 8>(x, lane);
    sort_steps<32, 16>(x, lane);
    sort_steps<64, 32>(x, lane);
    return x;
}

__device__ __forceinline__ float wave_sum(float x) {
    x += across<1>(x);
    x += across<2>(x);
    x += across<4>(x);
    x += across<8>(x);
    x += across<16>(x);
    return x + across<32>(x);
}

// exp(d) for d <= 0, to 2^-22 of it and the rounding of d's product
__device__ __forceinline__ float exp_below(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504f); }

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
// absent, and missing places get {-infinity, kNone}.  index(e): the index of x[e];
// no two are alike.  sorted: wave_sort of the threads' largest, top the thread's.
//
// The n-th largest of a wave's 64 lane maxima bounds the n-th best value from
// below, and so does the largest of the waves' bounds: what is below it is out.
// The rest, n and a few more, is listed and each entry put at its rank.  Values
// that are equal many times over can overrun the list; then the best are taken
// out one by one instead.
template <int E, typename Index>
__device__ __forceinline__ void block_best(const float (&x)[E], Index index, float top, float sorted, int n,
                                           BestShared &sh, Best *out) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float nth = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sorted), n - 1));
    if (lane == 0) sh.bound[wave] = nth;
    if (tid == 0) sh.count = 0;
    if (tid < n) out[tid] = {kNever, kNone};
    __syncthreads();
    float bound = sh.bound[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) bound = fmaxf(bound, sh.bound[w]);
    bound = fmaxf(bound, kLowest);  // -infinity does not pass
    if (top >= bound) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (x[e] >= bound) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kList) sh.list[at] = {x[e], index(e)};
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
            for (int e = 0; e < E; ++e) {
                const int i = index(e);
                if (before(lx, li, x[e], i) && x[e] > kNever && before(x[e], i, bx, bi)) {
                    bx = x[e];
                    bi = i;
                }
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

struct SelectPlan {
    int each;                          // logits of a thread: a segment has 256 times as many
    int segs;                          // segments of a row
    size_t off_stat, off_best, bytes;  // float2 [rows][segs] (max, sum); Best [groups][select][beams][segs]
};

// Segments of 8192 logits where that gives two workgroups a CU, else of 2048.
// (A row starts up to 7 elements into its first 16 bytes.)
SelectPlan select_plan(int64_t groups, int64_t beams, int64_t vocab, int64_t select) {
    SelectPlan p;
    p.each = groups * beams * ((vocab + 8191) / 8192) >= 512 ? 32 : 8;
    p.segs = (int)((vocab + 7 + kThreads * p.each - 1) / (kThreads * p.each));
    p.off_stat = 0;
    p.off_best = ((size_t)(groups * beams * p.segs) * sizeof(float2) + 255) / 256 * 256;
    p.bytes = p.off_best + (size_t)(groups * beams * p.segs * select) * sizeof(Best);
    return p;
}

// One workgroup a segment of a row: 16 bytes a thread and load, E logits in
// registers, read once.  Bound by that read.  (Places in a row are int: the last
// segment ends less than 2^14 past the row, and vocab is below 2^31 - 2^14.)
template <int ACT, int E>
__global__ __launch_bounds__(kThreads) void beam_segment_kernel(BeamSelectArgs a, SelectPlan p) {
    using T = typename Act<ACT>::T;
    constexpr int EB = Act<ACT>::kBytes, PER = 16 / EB;
    __shared__ BestShared sh;
    __shared__ Best best[kMaxSelect];
    __shared__ float2 stat[kWaves];
    const int row = (int)(blockIdx.x / (unsigned)p.segs), seg = (int)blockIdx.x - row * p.segs;
    const int tid = threadIdx.x, n = (int)a.select, V = (int)a.vocab;
    // a beam that has ended or is not alive has no continuation of its own here
    if (a.scores[row] == kNever || (a.finished && a.finished[row])) return;
    const T *x = static_cast<const T *>(a.logits) + (int64_t)row * a.ld;
    // from the 16 bytes that the row starts in
    const int base = seg * (kThreads * E) - (int)(reinterpret_cast<uintptr_t>(x) % 16) / EB;
    const auto index = [&](int e) { return base + (e / PER * kThreads + tid) * PER + e % PER; };
    float val[E];
#pragma unroll
    for (int e = 0; e < E; e += PER) {
        const int i = index(e);
        if (i >= 0 && i + PER <= V) {
            const uint4 w = *reinterpret_cast<const uint4 *>(x + i);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < PER; ++j)
                val[e + j] = ACT == kBF16 ? (j & 1 ? bf16_hi(u[j / 2]) : bf16_lo(u[j / 2])) : __uint_as_float(u[j % 4]);
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) val[e + j] = i + j >= 0 && i + j < V ? Act<ACT>::ld(x + i + j) : kNever;
        }
    }
    float top = kNever;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        val[e] = val[e] == val[e] ? val[e] : kNever;
        top = fmaxf(top, val[e]);
    }
    const float sorted = wave_sort(top);
    const float high = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(sorted)));
    float sum = 0.f;
    if (high == __builtin_inff()) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum += val[e] == high ? 1.f : 0.f;
    } else if (high > kNever) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum += exp_below(val[e] - high);
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) stat[tid >> 6] = make_float2(high, sum);
    block_best<E>(val, index, top, sorted, n, sh, best);
    if (tid == 0) {
        float m = kNever, s = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = fmaxf(m, stat[w].x);
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            if (stat[w].x > kNever) s += stat[w].x == m ? stat[w].y : stat[w].y * exp_below(stat[w].x - m);
        reinterpret_cast<float2 *>(a.ws + p.off_stat)[(int64_t)row * p.segs + seg] = make_float2(m, s);
    }
    const int K = (int)a.beams, g = row / K;
    if (tid < n)
        reinterpret_cast<Best *>(a.ws + p.off_best)[((int64_t)(g * n + tid) * K + (row - g * K)) * p.segs + seg] = best[tid];
}

// ------------------------------------------------------------------ groups

constexpr int kPickE = 12;  // candidates of a thread at a time (8: 16.1 us for 8 beams x 17 segments x 16, 12: 12.4)

// One workgroup a group.  What the segments handed on is taken rank by rank, all
// segments' first ones first, so that the leads spread over the lanes and
// block_best's bound is a tight one.
__global__ __launch_bounds__(kThreads) void beam_pick_kernel(BeamSelectArgs a, SelectPlan p) {
    __shared__ BestShared sh;
    __shared__ Best best[kMaxSelect];
    __shared__ float score0[kMaxSelect], top[kMaxSelect], lse[kMaxSelect];  // lse: log of the sum, after the maximum
    __shared__ bool ended[kMaxSelect];
    const int64_t g = blockIdx.x;
    const int tid = threadIdx.x, K = (int)a.beams, n = (int)a.select, V = (int)a.vocab;
    const unsigned lists = (unsigned)(K * p.segs), total = lists * n;
    const float2 *stat = reinterpret_cast<const float2 *>(a.ws + p.off_stat) + g * lists;
    const Best *cand = reinterpret_cast<const Best *>(a.ws + p.off_best) + g * total;
    Best have[kPickE];
    auto fetch = [&](unsigned c0) {
#pragma unroll
        for (int e = 0; e < kPickE; ++e) {
            const unsigned c = c0 + e * kThreads + tid;
            if (c < total) have[e] = cand[c];
        }
    };
    fetch(0);
    // four lanes a beam, each over every fourth segment, all beams at once
    if (const int k = tid >> 2; k < K) {
        const float s = a.scores[g * K + k];
        const bool f = a.finished && a.finished[g * K + k];
        float m = kNever, sum = 0.f;
        if (!f && s > kNever)
            for (int i = tid & 3; i < p.segs; i += 4) {
                const float2 st = stat[k * p.segs + i];
                if (st.x > m) {
                    sum = sum * exp_below(m - st.x) + st.y;
                    m = st.x;
                } else if (st.x > kNever) {
                    sum += st.x == m ? st.y : st.y * exp_below(st.x - m);
                }
            }
        float all = fmaxf(m, across<1>(m));
        all = fmaxf(all, across<2>(all));
        if (m != all) sum = m > kNever ? sum * exp_below(m - all) : 0.f;
        sum += across<1>(sum);
        sum += across<2>(sum);
        if ((tid & 3) == 0) {
            score0[k] = s;
            ended[k] = f;
            top[k] = all;
            lse[k] = logf(sum);
        }
    }
    if (tid < kMaxSelect) best[tid] = {kNever, kNone};
    __syncthreads();
    float val[kPickE + 1];
    int idx[kPickE + 1];
    for (unsigned c0 = 0; c0 < total; c0 += kThreads * kPickE) {
        if (c0 > 0) fetch(c0);
        float high = kNever;
#pragma unroll
        for (int e = 0; e < kPickE; ++e) {
            const unsigned c = c0 + e * kThreads + tid;
            val[e] = kNever;
            idx[e] = kNone;
            if (c < total) {
                const unsigned list = c % lists, k = list / (unsigned)p.segs;
                if (ended[k]) {  // one continuation, in the place of the beam's first
                    if (c == k * p.segs) {
                        val[e] = score0[k];
                        idx[e] = (int)k * V + (int)a.end_token;
                    }
                } else if (score0[k] > kNever && have[e].i != kNone) {
                    const float d = have[e].x == top[k] ? 0.f : have[e].x - top[k];
                    val[e] = score0[k] + (d - lse[k]);
                    idx[e] = (int)k * V + have[e].i;
                }
            }
            high = fmaxf(high, val[e]);
        }
        // the best so far stay in
        val[kPickE] = tid < n ? best[tid].x : kNever;
        idx[kPickE] = tid < n ? best[tid].i : kNone;
        high = fmaxf(high, val[kPickE]);
        __syncthreads();
        block_best<kPickE + 1>(val, [&](int e) { return idx[e]; }, high, wave_sort(high), n, sh, best);
    }
    // fewer than n continuations: the first others, all of score -infinity
    if (tid == 0 && best[n - 1].i == kNone) {
        int found = 0;
        while (found < n && best[found].i != kNone) ++found;
        for (int at = found, f = 0; at < n; ++f) {
            bool taken = false;
            for (int j = 0; j < found; ++j) taken |= best[j].i == f;
            if (!taken) best[at++].i = f;
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

constexpr int kMoves = 4;  // pieces of a row that a thread moves, one after the other (1: 489 us for 312, 2: 323, 8: 311)

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

// MOST: beams that pieces of this size are used for
template <typename T, int MOST>
void launch_reorder(const ReorderArgs &a, int64_t groups, hipStream_t stream) {
    const dim3 grid((unsigned)a.first[a.n], (unsigned)groups);
    // registers for a piece of every beam
    if (a.beams <= 8)
        beam_reorder_kernel<T, 8><<<grid, kThreads, 0, stream>>>(a);
    else if (a.beams <= 16)
        beam_reorder_kernel<T, 16><<<grid, kThreads, 0, stream>>>(a);
    else if constexpr (MOST > 16) {
        if (a.beams <= 32)
            beam_reorder_kernel<T, 32><<<grid, kThreads, 0, stream>>>(a);
        else if constexpr (MOST > 32)
            beam_reorder_kernel<T, 64><<<grid, kThreads, 0, stream>>>(a);
    }
}

}  // namespace

size_t beam_select_workspace(int64_t groups, int64_t beams, int64_t vocab, int64_t select) {
    return select_plan(groups, beams, vocab, select).bytes;
}

hipError_t launch_beam_select(const BeamSelectArgs &a, hipStream_t stream) {
    const SelectPlan p = select_plan(a.groups, a.beams, a.vocab, a.select);
    const dim3 grid((unsigned)(a.groups * a.beams * p.segs));
    if (p.each == 8) {
        if (a.act == kBF16)
            beam_segment_kernel<kBF16, 8><<<grid, kThreads, 0, stream>>>(a, p);
        else
            beam_segment_kernel<kF32, 8><<<grid, kThreads, 0, stream>>>(a, p);
    } else if (a.act == kBF16) {
        beam_segment_kernel<kBF16, 32><<<grid, kThreads, 0, stream>>>(a, p);
    } else {
        beam_segment_kernel<kF32, 32><<<grid, kThreads, 0, stream>>>(a, p);
    }
    beam_pick_kernel<<<dim3((unsigned)a.groups), kThreads, 0, stream>>>(a, p);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(int64_t groups, int64_t beams, const int32_t *parents, int64_t n, void *const *buffers,
                               const int64_t *row_bytes, hipStream_t stream) {
    if (beams == 1) return hipSuccess;
    // buffers of one piece size share a launch: 16 bytes where all rows allow it (8
    // for more than 16 beams, 4 for more than 32: a thread holds a piece of each),
    // else 4, else 1
    const int widest = beams <= 16 ? 16 : beams <= 32 ? 8 : 4;
    for (int size : {16, 8, 4, 1}) {
        if (size > widest || (size == 8 && widest == 16)) continue;
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
            // (a launch has fewer than 2^24 workgroups, a buffer at most 2^23)
            if (a.n == kBuffers || a.first[a.n] >= 1 << 23 || (i == n && a.n > 0)) {
                switch (size) {
                    case 16: launch_reorder<u32x4, 16>(a, groups, stream); break;
                    case 8: launch_reorder<u32x2, 32>(a, groups, stream); break;
                    case 4: launch_reorder<uint32_t, 64>(a, groups, stream); break;
                    default: launch_reorder<uint8_t, 64>(a, groups, stream);
                }
                const hipError_t err = hipGetLastError();
                if (err != hipSuccess) return err;
                a.n = 0;
            }
        }
    }
    return hipSuccess;
}

}  // namespace hm
