// drafts.hip -- verification of drafted tokens against the target's probabilities.
//
// Draft i is kept while u_i q_i(x_i) < p_i(x_i) (products of two float32 are exact in
// float64).  Behind the kept ones a token is drawn from the weights max(p - q, 0) of
// that place, or p's: the first whose cumulated weight exceeds u times the whole.
//
// A row of weights is cut into segments.  The first kernel, one workgroup a segment,
// finds the place and sums the segment in float64; the second, one workgroup a
// sequence, finds the segment that the number falls on, reads it again and finds the
// token in it.
#include "hm_internal.hpp"

namespace hm {
namespace {

constexpr int kThreads = 256, kEach = 16, kSegment = kThreads * kEach;

__device__ __forceinline__ float weighed(float p) { return p > 0.0f && p < __builtin_inff() ? p : 0.0f; }

// The place behind the kept drafts of sequence b; refused: a draft stands there.
template <int ACT>
__device__ __forceinline__ int place_of(const VerifyArgs &a, int64_t b, bool &refused) {
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
    const uint64_t gone = ~__ballot(kept);  // a lane past n is not kept
    const int place = gone ? __builtin_ctzll(gone) : kWave;
    refused = place < n;
    return place;
}

// The weights of sequence b's place.
template <int ACT> struct Weights {
    using A = Act<ACT>;
    using T = typename A::T;
    const T *p, *q;  // q null: none, or one token's
    int out;         // a draft without chance that was refused, else -1
    bool rest;       // max(p - q, 0)
    __device__ Weights(const VerifyArgs &a, int64_t b, int place, bool refused) {
        p = static_cast<const T *>(a.p) + (b * (a.T + 1) + place) * a.ld_p;
        q = refused && a.q ? static_cast<const T *>(a.q) + (b * a.T + place) * a.ld_q : nullptr;
        out = refused && !a.q ? a.tokens[b * a.T + place] : -1;
        rest = refused;
    }
    __device__ double all(int64_t v) const { return weighed(A::ld(p + v)); }
    __device__ double left(int64_t v, double all) const {
        if (q) {
            const double d = all - (double)weighed(A::ld(q + v));
            return d > 0.0 ? d : 0.0;
        }
        return v == out ? 0.0 : all;
    }
};

__device__ __forceinline__ double block_sum(double x, double *sh) {
    for (int s = 32; s > 0; s >>= 1) x += __shfl_xor(x, s);
    __syncthreads();
    if (threadIdx.x % kWave == 0) sh[threadIdx.x / kWave] = x;
    __syncthreads();
    return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

template <int ACT>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(VerifyArgs a, int segs) {
    __shared__ double sh[4];
    const int64_t b = blockIdx.x / segs, seg = blockIdx.x % segs;
    bool refused;
    const int place = place_of<ACT>(a, b, refused);
    const Weights<ACT> w(a, b, place, refused);
    double left = 0.0, all = 0.0;
    for (int e = 0; e < kEach; ++e) {
        const int64_t v = seg * kSegment + e * kThreads + threadIdx.x;
        if (v >= a.V) break;
        const double x = w.all(v);
        all += x;
        left += w.left(v, x);
    }
    left = block_sum(left, sh);
    all = block_sum(all, sh);
    if (threadIdx.x == 0) {
        double *out = reinterpret_cast<double *>(a.ws) + 2 * (b * segs + seg);
        out[0] = left;
        out[1] = all;
    }
}

template <int ACT>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(VerifyArgs a, int segs) {
    __shared__ double weights[kSegment], sums[kThreads];
    __shared__ int found, last;
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x;
    bool refused;
    const int place = place_of<ACT>(a, b, refused);
    const Weights<ACT> w(a, b, place, refused);
    const double *part = reinterpret_cast<const double *>(a.ws) + 2 * b * segs;
    // every thread alike: few segments
    double whole = 0.0;
    bool rest = refused;
    for (int s = 0; s < segs; ++s) whole += part[2 * s];
    if (!(whole > 0.0)) {
        rest = false;
        whole = 0.0;
        for (int s = 0; s < segs; ++s) whole += part[2 * s + 1];
    }
    int token = -1;
    if (whole > 0.0) {
        const double at = (double)a.u[b * (a.T + 1) + a.T] * whole;
        double before = 0.0, sum = 0.0;
        int seg = -1;
        for (int s = 0; s < segs; ++s) {
            const double x = part[2 * s + !rest];
            if (x > 0.0) {  // the last one that has weight, where rounding leaves none
                seg = s;
                before = sum;
            }
            sum += x;
            if (x > 0.0 && sum > at) break;
        }
        for (int e = 0; e < kEach; ++e) {
            const int i = e * kThreads + tid;
            const int64_t v = (int64_t)seg * kSegment + i;
            const double x = v < a.V ? w.all(v) : 0.0;
            weights[i] = v < a.V && rest ? w.left(v, x) : x;
        }
        if (tid == 0) {
            found = kSegment;
            last = -1;
        }
        __syncthreads();
        double mine = 0.0;
        for (int e = 0; e < kEach; ++e) mine += weights[tid * kEach + e];
        sums[tid] = mine;
        __syncthreads();
        for (int t = 0; t < tid; ++t) before += sums[t];
        for (int e = 0; e < kEach; ++e) {
            const double x = weights[tid * kEach + e];
            before += x;
            if (x > 0.0) {
                atomicMax(&last, tid * kEach + e);
                if (before > at) {
                    atomicMin(&found, tid * kEach + e);
                    break;
                }
            }
        }
        __syncthreads();
        token = seg * kSegment + (found < kSegment ? found : last);
    }
    if (tid <= a.T)
        a.out_tokens[b * (a.T + 1) + tid] = tid < place ? a.tokens[b * a.T + tid] : tid == place ? token : -1;
    if (tid == 0) a.out_accepted[b] = place;
}

int segments(int64_t V) { return (int)((V + kSegment - 1) / kSegment); }

}  // namespace

size_t draft_verify_workspace(int64_t B, int64_t V) { return (size_t)B * (size_t)segments(V) * 2 * sizeof(double); }

hipError_t launch_draft_verify(const VerifyArgs &a, hipStream_t stream) {
    const int segs = segments(a.V);
    const dim3 grid((unsigned)(a.B * segs)), rows((unsigned)a.B);
    if (a.act == kBF16) {
        verify_sums_kernel<kBF16><<<grid, kThreads, 0, stream>>>(a, segs);
        verify_draw_kernel<kBF16><<<rows, kThreads, 0, stream>>>(a, segs);
    } else {
        verify_sums_kernel<kF32><<<grid, kThreads, 0, stream>>>(a, segs);
        verify_draw_kernel<kF32><<<rows, kThreads, 0, stream>>>(a, segs);
    }
    return hipGetLastError();
}

}  // namespace hm
