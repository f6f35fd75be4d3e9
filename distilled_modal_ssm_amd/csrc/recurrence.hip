// recurrence.hip -- gated recurrence: h_t = f_t h_{t-1} + i_t v_t, y_t = q_t h_t,
// over a prompt, for one token, and backward.
//
// One lane a channel, token after token.  Backward, chunk after chunk from the
// last: h is formed again from the chunk's first state, then
//     dh_t = q_t dy_t + f_{t+1} dh_{t+1},
//     dq_t = dy_t h_t,  dv_t = i_t dh_t,  dg_t = dh_t (f' h_{t-1} + i' v_t).
#include "hm_internal.hpp"

namespace hm {
namespace {

// f and i of a gate g; away = 1 - f without cancellation.  f is rounded from
// 1 - away where it is over 1/2, so that slow channels keep half a rounding.
template <int GATE, int INPUT>
__device__ __forceinline__ void gate_of(float g, float &f, float &i) {
    float away;
    if constexpr (GATE == kGateLog) {
        if (fabsf(g) < 0.35f) {  // -expm1(g) by its series, to 0.35^7 / 8! = 2^-26
            float s = fmaf(g, 1.0f / 5040, 1.0f / 720);
            s = fmaf(g, s, 1.0f / 120);
            s = fmaf(g, s, 1.0f / 24);
            s = fmaf(g, s, 1.0f / 6);
            s = fmaf(g, s, 0.5f);
            away = -fmaf(g * g, s, g);
            f = 1.0f - away;
        } else {
            f = __builtin_amdgcn_exp2f(g * 1.44269504f);
            away = 1.0f - f;
        }
    } else {
        const float e = __builtin_amdgcn_exp2f(fabsf(g) * -1.44269504f);
        const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
        f = g < 0.0f ? small : 1.0f - small;
        away = g < 0.0f ? 1.0f - small : small;
    }
    if constexpr (INPUT == kInputFree) i = 1.0f;
    if constexpr (INPUT == kInputConvex) i = away;
    if constexpr (INPUT == kInputNorm) i = __builtin_amdgcn_sqrtf(fmaxf(away * (1.0f + f), 0.0f));
}

// and the derivatives of both by g
template <int GATE, int INPUT>
__device__ __forceinline__ void gate_grad(float g, float &f, float &i, float &df, float &di) {
    gate_of<GATE, INPUT>(g, f, i);
    if constexpr (GATE == kGateLog) {
        df = f;
        di = INPUT == kInputFree ? 0.0f : INPUT == kInputConvex ? -f : i > 0.0f ? -f * f * __builtin_amdgcn_rcpf(i) : 0.0f;
    } else {
        float h, away;
        gate_of<GATE, kInputConvex>(g, h, away);
        df = f * away;
        di = INPUT == kInputFree ? 0.0f : INPUT == kInputConvex ? -df : -f * f * i * __builtin_amdgcn_rcpf(1.0f + f);
    }
}

__device__ __forceinline__ int64_t row_length(const RecurArgs &a, int64_t b) {
    if (!a.lengths) return a.L;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

template <int ACT, int GATE, int INPUT>
__global__ __launch_bounds__(64) void recurrence_kernel(RecurArgs a) {
    using A = Act<ACT>;
    using T = typename A::T;
    const int64_t tiles = (a.D + 63) / 64, b = blockIdx.x / tiles, c = blockIdx.x % tiles * 64 + threadIdx.x;
    if (c >= a.D) return;
    const int64_t n = row_length(a, b), chunks = (a.L + kRecurChunk - 1) / kRecurChunk;
    float h = a.state_in ? a.state_in[b * a.D + c] : 0.0f;
    for (int64_t t = 0; t < a.L; ++t) {
        const int64_t r = b * a.L + t;
        float y = 0.0f;
        if (t < n) {
            if (a.chunk_states && t % kRecurChunk == 0) a.chunk_states[(b * chunks + t / kRecurChunk) * a.D + c] = h;
            float f, i;
            gate_of<GATE, INPUT>(A::ld(static_cast<const T *>(a.g) + r * a.ld_g + c), f, i);
            h = fmaf(f, h, i * A::ld(static_cast<const T *>(a.v) + r * a.ld_v + c));
            y = a.q ? h * A::ld(static_cast<const T *>(a.q) + r * a.ld_q + c) : h;
        }
        A::st(static_cast<T *>(a.y) + r * a.ld_y + c, y);
    }
    a.state_out[b * a.D + c] = h;
}

template <int ACT, int GATE, int INPUT>
__global__ __launch_bounds__(64) void recurrence_backward_kernel(RecurArgs a) {
    using A = Act<ACT>;
    using T = typename A::T;
    __shared__ float hs[kRecurChunk][64];
    const int lane = threadIdx.x;
    const int64_t tiles = (a.D + 63) / 64, b = blockIdx.x / tiles, c = blockIdx.x % tiles * 64 + lane;
    if (c >= a.D) return;
    const int64_t n = row_length(a, b), chunks = (a.L + kRecurChunk - 1) / kRecurChunk;
    const T *q = static_cast<const T *>(a.q) + c, *g = static_cast<const T *>(a.g) + c;
    const T *v = static_cast<const T *>(a.v) + c, *dy = static_cast<const T *>(a.dy) + c;
    T *dq = static_cast<T *>(a.dq) + c, *dg = static_cast<T *>(a.dg) + c, *dv = static_cast<T *>(a.dv) + c;
    for (int64_t t = n; t < a.L; ++t) {
        const int64_t r = b * a.L + t;
        if (a.q) A::st(dq + r * a.ld_dq, 0.0f);
        A::st(dg + r * a.ld_dg, 0.0f);
        A::st(dv + r * a.ld_dv, 0.0f);
    }
    float back = a.dstate_out ? a.dstate_out[b * a.D + c] : 0.0f;
    for (int64_t k = (n + kRecurChunk - 1) / kRecurChunk - 1; k >= 0; --k) {
        const int64_t t0 = k * kRecurChunk, t1 = t0 + kRecurChunk < n ? t0 + kRecurChunk : n;
        const float first = a.chunk_states[(b * chunks + k) * a.D + c];
        float h = first;
        for (int64_t t = t0; t < t1; ++t) {
            const int64_t r = b * a.L + t;
            float f, i;
            gate_of<GATE, INPUT>(A::ld(g + r * a.ld_g), f, i);
            h = fmaf(f, h, i * A::ld(v + r * a.ld_v));
            hs[t - t0][lane] = h;
        }
        for (int64_t t = t1 - 1; t >= t0; --t) {
            const int64_t r = b * a.L + t;
            float f, i, df, di;
            gate_grad<GATE, INPUT>(A::ld(g + r * a.ld_g), f, i, df, di);
            const float vt = A::ld(v + r * a.ld_v), dyt = A::ld(dy + r * a.ld_dy);
            const float before = t > t0 ? hs[t - t0 - 1][lane] : first;
            float dh = back + dyt;
            if (a.q) {
                A::st(dq + r * a.ld_dq, dyt * hs[t - t0][lane]);
                dh = fmaf(dyt, A::ld(q + r * a.ld_q), back);
            }
            A::st(dg + r * a.ld_dg, dh * fmaf(df, before, di * vt));
            A::st(dv + r * a.ld_dv, dh * i);
            back = f * dh;
        }
    }
    if (a.dstate_in) a.dstate_in[b * a.D + c] = back;
}

template <int ACT, int GATE, int INPUT>
__global__ __launch_bounds__(256) void recurrence_token_kernel(RecurArgs a) {
    using A = Act<ACT>;
    using T = typename A::T;
    const int64_t tiles = (a.D + 255) / 256, b = blockIdx.x / tiles, c = blockIdx.x % tiles * 256 + threadIdx.x;
    if (c >= a.D) return;
    int64_t from = b;
    if (a.src_rows) {
        const int64_t r = a.src_rows[b];
        if (r >= 0 && r < a.B) from = r;
    }
    float f, i;
    gate_of<GATE, INPUT>(A::ld(static_cast<const T *>(a.g) + b * a.ld_g + c), f, i);
    const float h = fmaf(f, a.state_in[from * a.D + c], i * A::ld(static_cast<const T *>(a.v) + b * a.ld_v + c));
    a.state_out[b * a.D + c] = h;
    A::st(static_cast<T *>(a.y) + b * a.ld_y + c, a.q ? h * A::ld(static_cast<const T *>(a.q) + b * a.ld_q + c) : h);
}

// A launch of the kernel for the call's types.
template <typename F> hipError_t for_types(const RecurArgs &a, F launch) {
    auto input = [&](auto act, auto gate) {
        if (a.input == kInputFree) launch(act, gate, std::integral_constant<int, kInputFree>{});
        else if (a.input == kInputConvex) launch(act, gate, std::integral_constant<int, kInputConvex>{});
        else launch(act, gate, std::integral_constant<int, kInputNorm>{});
    };
    auto gate = [&](auto act) {
        if (a.gate == kGateLog) input(act, std::integral_constant<int, kGateLog>{});
        else input(act, std::integral_constant<int, kGateSigmoid>{});
    };
    if (a.act == kBF16) gate(std::integral_constant<int, kBF16>{});
    else gate(std::integral_constant<int, kF32>{});
    return hipGetLastError();
}

}  // namespace

size_t recurrence_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_recurrence_prefill(const RecurArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.D + 63) / 64)));
    return for_types(a, [&](auto act, auto gate, auto input) {
        recurrence_kernel<decltype(act)::value, decltype(gate)::value, decltype(input)::value><<<grid, 64, 0, stream>>>(a);
    });
}

hipError_t launch_recurrence_backward(const RecurArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.D + 63) / 64)));
    return for_types(a, [&](auto act, auto gate, auto input) {
        recurrence_backward_kernel<decltype(act)::value, decltype(gate)::value, decltype(input)::value><<<grid, 64, 0, stream>>>(a);
    });
}

hipError_t launch_recurrence_decode(const RecurArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.D + 255) / 256)));
    return for_types(a, [&](auto act, auto gate, auto input) {
        recurrence_token_kernel<decltype(act)::value, decltype(gate)::value, decltype(input)::value><<<grid, 256, 0, stream>>>(a);
    });
}

}  // namespace hm
