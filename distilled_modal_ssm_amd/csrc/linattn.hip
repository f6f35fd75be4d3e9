// linattn.hip -- linear attention with a decay: the recurrence over a prompt
// and for one generated token.  Per batch row and head, S [dk][dv]:
//     S_t = exp(a_t) S_{t-1} + k_t v_t^T,      y_t = scale * S_t^T q_t.
#include "hm_internal.hpp"

namespace hm {
namespace {

constexpr int kThreads = 256;

// exp(a) of a log decay; a is bounded below so that sums of it stay finite
__device__ __forceinline__ float bound_decay(float a) { return a < -1000.f ? -1000.f : a; }

// ------------------------------------------------------------------ prompt

constexpr int kTok = 16;   // tokens staged at a time
constexpr int kCols = 64;  // value columns of a workgroup, one a lane
constexpr int kRows = 64;  // key rows of a wave: four waves cover 256

// One workgroup for a batch row, head and 64 value columns: token after token,
// lane = column, wave = 64 key rows whose state the lane holds in registers.
template <int ACT>
__global__ __launch_bounds__(kThreads) void linattn_scan_kernel(LinAttnArgs a) {
    using T = typename Act<ACT>::T;
    __shared__ float qs[kTok][256], ks[kTok][256], vs[kTok][kCols], as[kTok], part[4][kTok][kCols];
    const int64_t b = blockIdx.x / a.s.H, h = blockIdx.x - b * a.s.H;
    const int v0 = blockIdx.y * kCols, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int dk = a.s.dk, dv = a.s.dv, col = v0 + lane;
    const T *q = static_cast<const T *>(a.q) + b * a.L * a.ld_q + h * a.s.qh / a.s.H * dk;
    const T *k = static_cast<const T *>(a.k) + b * a.L * a.ld_k + h * a.s.kh / a.s.H * dk;
    const T *v = static_cast<const T *>(a.v) + b * a.L * a.ld_v + h * a.s.vh / a.s.H * dv;
    T *y = static_cast<T *>(a.y) + b * a.L * a.ld_y + h * dv;
    const int64_t sbase = (b * a.s.H + h) * (int64_t)dk * dv;
    int64_t len = a.L;
    if (a.lengths) len = a.lengths[b] < 0 ? 0 : a.lengths[b] < a.L ? a.lengths[b] : a.L;
    float S[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = wave * kRows + i;
        S[i] = a.state_in && row < dk && col < dv ? a.state_in[sbase + (int64_t)row * dv + col] : 0.f;
    }
    for (int64_t t0 = 0; t0 < a.L; t0 += kTok) {
        __syncthreads();
        for (int i = tid; i < kTok * 256; i += kThreads) {
            const int t = i / 256, c = i % 256;
            const bool in = t0 + t < len && c < dk;
            qs[t][c] = in ? Act<ACT>::ld(q + (t0 + t) * a.ld_q + c) : 0.f;
            ks[t][c] = in ? Act<ACT>::ld(k + (t0 + t) * a.ld_k + c) : 0.f;
            if (c < kCols)
                vs[t][c] = t0 + t < len && v0 + c < dv ? Act<ACT>::ld(v + (t0 + t) * a.ld_v + v0 + c) : 0.f;
            if (c == 0) {
                float d = 0.f;
                if (a.decay && t0 + t < len)
                    d = a.decay[a.ld_decay ? (b * a.L + t0 + t) * a.ld_decay + h : h];
                as[t] = expf(bound_decay(d));
            }
        }
        __syncthreads();
        for (int t = 0; t < kTok; ++t) {
            float o = 0.f;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                S[i] = fmaf(as[t], S[i], ks[t][wave * kRows + i] * vs[t][lane]);
                o = fmaf(qs[t][wave * kRows + i], S[i], o);
            }
            part[wave][t][lane] = o;
        }
        __syncthreads();
        for (int i = tid; i < kTok * kCols; i += kThreads) {
            const int t = i / kCols, c = i % kCols;
            if (t0 + t < a.L && v0 + c < dv)
                Act<ACT>::st(y + (t0 + t) * a.ld_y + v0 + c,
                             a.s.scale * (part[0][t][c] + part[1][t][c] + part[2][t][c] + part[3][t][c]));
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = wave * kRows + i;
        if (row < dk && col < dv) a.state_out[sbase + (int64_t)row * dv + col] = S[i];
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

}  // namespace

size_t linattn_workspace(const LinAttnShape &, int64_t) { return 0; }

hipError_t launch_linattn_prefill(const LinAttnArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.s.B * a.s.H), (unsigned)((a.s.dv + kCols - 1) / kCols));
    if (a.s.act == kBF16)
        linattn_scan_kernel<kBF16><<<grid, kThreads, 0, stream>>>(a);
    else
        linattn_scan_kernel<kF32><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
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
