// drafts.hip -- verification of drafted tokens against the target's probabilities.
//
// Draft i is kept while u_i q_i(x_i) < p_i(x_i) (products of two float32 are exact in
// float64).  Behind the kept ones a token is drawn from the weights max(p - q, 0) of
// that place, or p's: the first whose cumulated weight exceeds u times the whole.
//
// A row of weights is cut into parts of 1024.  The first kernel, a wave a part, finds the
// place and sums the part in float64; the second, one workgroup a sequence, finds the
// part that the number falls on from the sums, reads it again and finds the token in it.
// Vocabularies of up to four parts take one kernel that does both (4000 tokens: 6.5 us for
// one sequence and 7.2 for 256, 7.6 and 9.2 in two; of 8 parts, by 16 waves: 9.9, 8.1).
// What bounds it: launches and memory latency; a large batch's first kernel, HBM (64 x
// 131072 float32 with q: 12.2 us, 5 TB/s).
// Sums are in float64 because which token a number falls on is a matter of the last
// digits, and in a fixed order.
#include "hm_internal.hpp"

namespace hm {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kPart = 1024, kEach = kPart / kWave;

// Probabilities that are none count as 0.
__device__ __forceinline__ float weighed(float p) { return p > 0.0f && p < __builtin_inff() ? p : 0.0f; }

// The workspace: sums of max(p - q, 0) and of p over every part, and the places.
struct Work {
    double *left, *all;  // [B][parts]
    int *place;          // [B]; 256 more where a draft was refused
};
constexpr int kRefused = 256;

__host__ __device__ inline int64_t parts_of(int64_t V) { return (V + kPart - 1) / kPart; }

__device__ __forceinline__ Work work_of(const VerifyArgs &a, int64_t parts) {
    double *left = reinterpret_cast<double *>(a.ws);
    return {left, left + a.B * parts, reinterpret_cast<int *>(left + 2 * a.B * parts)};
}

// The place behind the kept drafts of sequence b, with kRefused where a draft stands there.
template <int ACT> __device__ __forceinline__ int place_of(const VerifyArgs &a, int64_t b) {
    using A = Act<ACT>;
    using T = typename A::T;
    int n = a.lengths ? a.lengths[b] : a.T;
    n = n < 0 ? 0 : n > a.T ? a.T : n;
    const int lane = threadIdx.x % kWave;
    bool kept = false;
    if (lane < n) {
        const int x = a.tokens[b * a.T + lane];
        if (x >= 0 && x < a.V) {
            const float p = weighed(A::ld(static_cast<const T *>(a.p) + (b * (a.T + 1) + lane) * a.ld_p + x));
            const float q = a.q ? weighed(A::ld(static_cast<const T *>(a.q) + (b * a.T + lane) * a.ld_q + x)) : 1.0f;
            kept = (double)a.u[b * (a.T + 1) + lane] * (double)q < (double)p;
        }
    }
    const int place = __builtin_ctzll(~__ballot(kept));  // a lane past n is not kept, and n < 64
    return place < n ? place | kRefused : place;
}

// The weights of sequence b's place.
template <int ACT> struct Weights {
    using A = Act<ACT>;
    using T = typename A::T;
    const T *p, *q;  // q null: none, or one token's
    int64_t out;     // a draft without chance that was refused, else -1
    __device__ Weights(const VerifyArgs &a, int64_t b, int state) {
        const int place = state % kRefused;
        const bool refused = state >= kRefused;
        p = static_cast<const T *>(a.p) + (b * (a.T + 1) + place) * a.ld_p;
        q = refused && a.q ? static_cast<const T *>(a.q) + (b * a.T + place) * a.ld_q : nullptr;
        out = refused && !a.q ? a.tokens[b * a.T + place] : -1;
    }
    // of token v, whose probabilities these are
    __device__ double left(int64_t v, float p, float q) const {
        const double d = (double)weighed(p) - (double)weighed(q);
        return v == out || d < 0.0 ? 0.0 : d;
    }
};

// A wave's values of a part: element k of a lane is 64 k + lane of it, or 128 k + 2 lane
// and the one behind where PAIRS of bfloat16 are aligned; past `count` they are 0.
template <int ACT, bool PAIRS> __device__ __forceinline__ void load_part(const void *row, int count, float (&x)[kEach]) {
    const int lane = threadIdx.x % kWave;
    const auto region = make_region(row, row ? count * Act<ACT>::kBytes : 0);
    if constexpr (PAIRS) {
#pragma unroll
        for (int k = 0; k < kEach / 2; ++k) {
            const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(region, 4 * (kWave * k + lane), 0, 0);
            x[2 * k] = bf16_lo(w);
            x[2 * k + 1] = bf16_hi(w);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kEach; ++k) x[k] = BufAct<ACT>::ld(region, Act<ACT>::kBytes * (kWave * k + lane), 0);
    }
}

// Sums over a part by a wave: of max(p - q, 0) and of p, in every lane.
template <int ACT, bool PAIRS>
__device__ __forceinline__ double2 sum_part(const VerifyArgs &a, const Weights<ACT> &w, int64_t part) {
    const int lane = threadIdx.x % kWave;
    const int64_t v0 = part * kPart;
    const int count = a.V - v0 < kPart ? (int)(a.V - v0) : kPart;
    float p[kEach], q[kEach];
    load_part<ACT, PAIRS>(w.p + v0, count, p);
    load_part<ACT, PAIRS>(w.q ? w.q + v0 : nullptr, count, q);
    double left = 0.0, all = 0.0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int at = PAIRS ? 2 * (kWave * (k / 2) + lane) + k % 2 : kWave * k + lane;
        left += w.left(v0 + at, p[k], q[k]);
        all += (double)weighed(p[k]);
    }
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) {
        left += __shfl_xor(left, s);
        all += __shfl_xor(all, s);
    }
    return make_double2(left, all);
}

template <int ACT, bool PAIRS>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(VerifyArgs a, int64_t parts) {
    const int64_t groups = (parts + kWaves - 1) / kWaves, b = blockIdx.x / groups;
    const int64_t part = blockIdx.x % groups * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (part >= parts) return;
    const int state = place_of<ACT>(a, b);
    const double2 sums = sum_part<ACT, PAIRS>(a, Weights<ACT>(a, b, state), part);
    if (threadIdx.x % kWave == 0) {
        const Work work = work_of(a, parts);
        work.left[b * parts + part] = sums.x;
        work.all[b * parts + part] = sums.y;
        if (part == 0) work.place[b] = state;
    }
}

// The sum of the threads' x before this one's, and the whole.
__device__ __forceinline__ double before_in_block(double x, double *sh, double &whole) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    double sum = x;
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) {
        const double other = __shfl_up(sum, s);
        if (lane >= s) sum += other;
    }
    __syncthreads();  // the last use of sh
    if (lane == kWave - 1) sh[wave] = sum;
    __syncthreads();
    const double up = __shfl_up(sum, 1);
    double before = lane > 0 ? up : 0.0;
    whole = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sh[w];
        whole += sh[w];
    }
    return before;
}

// Of all the workgroup's weights (a thread has n of them from `first` on, weight(i) the
// i-th), the first whose cumulated sum exceeds `at`, or where rounding leaves none the last
// that is above 0; -1 where all are 0.  before: the sum before the thread's weights; then
// the sum before the one found.
// (Lanes and waves are asked in order: as minima and maxima of all threads in the LDS it
// took 10 us.)
struct Found {
    int64_t over[kWaves], last[kWaves];  // of a wave, -1 where it has none
    double over_before[kWaves], last_before[kWaves], sums[kWaves];
};

template <typename F>
__device__ __forceinline__ int64_t find(int64_t first, int64_t n, F weight, double at, double &before, Found &sh) {
    int64_t over = -1, last = -1;
    double sum = before, over_before = 0.0, last_before = 0.0;
    for (int64_t i = 0; i < n; ++i) {
        const double x = weight(i);
        if (x > 0.0) {
            last = first + i;
            last_before = sum;
            if (sum + x > at) {
                over = first + i;
                over_before = sum;
                break;
            }
        }
        sum += x;
    }
    const uint64_t overs = __ballot(over >= 0), lasts = __ballot(last >= 0);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    __syncthreads();  // the last use of sh
    if (lane == (overs ? __builtin_ctzll(overs) : 0)) {
        sh.over[wave] = over;
        sh.over_before[wave] = over_before;
    }
    if (lane == (lasts ? 63 - __builtin_clzll(lasts) : 0)) {
        sh.last[wave] = last;
        sh.last_before[wave] = last_before;
    }
    __syncthreads();
    int64_t found = -1;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        if (sh.last[w] >= 0) {
            found = sh.last[w];
            before = sh.last_before[w];
        }
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w)
        if (sh.over[w] >= 0) {
            found = sh.over[w];
            before = sh.over_before[w];
        }
    return found;
}

// The token of sequence b from its parts' sums, and its outputs.
template <int ACT>
__device__ __forceinline__ void draw(const VerifyArgs &a, int64_t b, int state, const Weights<ACT> &w, const double *left,
                                     const double *all, int64_t parts, Found &sh) {
    using A = Act<ACT>;
    constexpr int kMine = kPart / kThreads;
    const int tid = threadIdx.x, place = state % kRefused;
    // the part; a thread has `each` neighbours
    const int64_t each = (parts + kThreads - 1) / kThreads, first = tid * each;
    const int64_t mine = first >= parts ? 0 : parts - first < each ? parts - first : each;
    bool rest = true;  // max(p - q, 0); p where that is 0 all over
    const double *part = left;
    double whole, before;
    for (;;) {
        double sum = 0.0;
        for (int64_t i = 0; i < mine; ++i) sum += part[first + i];
        before = before_in_block(sum, sh.sums, whole);
        if (whole > 0.0 || !rest) break;
        rest = false;
        part = all;
    }
    int64_t token = -1;
    if (whole > 0.0) {
        const double at = (double)a.u[b * (a.T + 1) + a.T] * whole;
        const int64_t found = find(first, mine, [&](int64_t i) { return part[first + i]; }, at, before, sh);
        const double so_far = before;
        // and the token in it: a thread has kMine neighbours
        const int64_t v0 = found * kPart + tid * kMine;
        double x[kMine], sum = 0.0;
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            const int64_t v = v0 + e;
            x[e] = 0.0;
            if (v < a.V) {
                const float p = A::ld(w.p + v);
                x[e] = rest ? w.left(v, p, w.q ? A::ld(w.q + v) : 0.0f) : (double)weighed(p);
            }
            sum += x[e];
        }
        double ignored;
        before = so_far + before_in_block(sum, sh.sums, ignored);
        token = find(v0, kMine, [&](int64_t i) { return x[i]; }, at, before, sh);
    }
    if (tid <= a.T)
        a.out_tokens[b * (a.T + 1) + tid] = tid < place ? a.tokens[b * a.T + tid] : tid == place ? (int)token : -1;
    if (tid == 0) a.out_accepted[b] = place;
}

template <int ACT>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, int64_t parts) {
    __shared__ Found sh;
    const int64_t b = blockIdx.x;
    const Work work = work_of(a, parts);
    const int state = work.place[b];
    draw<ACT>(a, b, state, Weights<ACT>(a, b, state), work.left + b * parts, work.all + b * parts, parts, sh);
}

template <int ACT, bool PAIRS> __global__ __launch_bounds__(kThreads) void verify_whole_kernel(VerifyArgs a, int parts) {
    __shared__ Found sh;
    __shared__ double left[kWaves], all[kWaves];
    const int64_t b = blockIdx.x;
    const int state = place_of<ACT>(a, b), part = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Weights<ACT> w(a, b, state);
    if (part < parts) {
        const double2 sums = sum_part<ACT, PAIRS>(a, w, part);
        if (threadIdx.x % kWave == 0) {
            left[part] = sums.x;
            all[part] = sums.y;
        }
    }
    __syncthreads();
    draw<ACT>(a, b, state, w, left, all, parts, sh);
}

template <int ACT, bool PAIRS> void launch(const VerifyArgs &a, hipStream_t stream) {
    const int64_t parts = parts_of(a.V);
    const dim3 grid((unsigned)(a.B * ((parts + kWaves - 1) / kWaves))), rows((unsigned)a.B);
    if (parts <= kWaves) {
        verify_whole_kernel<ACT, PAIRS><<<rows, kThreads, 0, stream>>>(a, (int)parts);
    } else {
        verify_sums_kernel<ACT, PAIRS><<<grid, kThreads, 0, stream>>>(a, parts);
        verify_draw_kernel<ACT><<<rows, kThreads, 0, stream>>>(a, parts);
    }
}

}  // namespace

size_t draft_verify_workspace(int64_t B, int64_t V) {
    return (size_t)B * ((size_t)parts_of(V) * 2 * sizeof(double) + sizeof(int));
}

hipError_t launch_draft_verify(const VerifyArgs &a, hipStream_t stream) {
    auto pairs = [&](const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0; };
    if (a.act == kF32) launch<kF32, false>(a, stream);
    else if (a.V % 2 == 0 && pairs(a.p, a.ld_p) && (!a.q || pairs(a.q, a.ld_q))) launch<kBF16, true>(a, stream);
    else launch<kBF16, false>(a, stream);
    return hipGetLastError();
}

}  // namespace hm
