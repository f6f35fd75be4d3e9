// recurrence.hip -- gated recurrence: h_t = f_t h_{t-1} + i_t v_t, y_t = q_t h_t,
// over a prompt, for one token, and backward.
//
// A run of tokens maps the h before it to the h behind it by h -> A h + H, A the
// product of its f; two runs join by (A1 A2, A2 H1 + H2).  A workgroup takes W x T
// tokens of a tile of channels, its wave w tokens w T .. of them, a lane one or two
// channels: tokens in registers, (A, H) of each wave through the LDS, of each
// workgroup through global memory, and then the recurrence once more from the h that
// came in.  So everything is read once.  Backward the same from the end, with
//     dh_t = q_t dy_t + b_t,   b_{t-1} = f_t dh_t      (b -> A b + K over a run)
// beside the h, formed again from what the prompt kept every 64 tokens.
//
// Workgroups join through slots of the workspace, (A, H) as one 64-bit word a
// channel, filled with a mark beforehand; a word that is not the mark is there.  A
// workgroup waits for up to kGroup words: its group's earlier workgroups and the h
// behind the group before.  Which words, and the order of the products, are fixed by
// its place, so results do not depend on timing.  Places go by a counter that each
// workgroup draws from when it starts, earlier runs first: whom it waits for has
// started, and needs nothing from later ones, so every wait ends.
#include "hm_internal.hpp"

namespace hm {
namespace {

constexpr int kGroup = 8;               // workgroups that join one by one
constexpr uint64_t kMark = ~0ull;       // a word that is not there yet

// ------------------------------------------------------------------ gates

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

// ------------------------------------------------------------------ a lane's channels

template <int ACT, int V> struct Lane;
template <> struct Lane<kBF16, 1> {
    using R = uint16_t;
    __device__ static void get(R r, float (&x)[1]) { x[0] = __uint_as_float((uint32_t)r << 16); }
    __device__ static R put(const float (&x)[1]) { return (uint16_t)f32_to_bf16(x[0]); }
};
template <> struct Lane<kBF16, 2> {
    using R = uint32_t;
    __device__ static void get(R r, float (&x)[2]) {
        x[0] = bf16_lo(r);
        x[1] = bf16_hi(r);
    }
    __device__ static R put(const float (&x)[2]) { return pack_bf16x2(x[0], x[1]); }
};
template <> struct Lane<kF32, 1> {
    using R = float;
    __device__ static void get(R r, float (&x)[1]) { x[0] = r; }
    __device__ static R put(const float (&x)[1]) { return x[0]; }
};
template <> struct Lane<kF32, 2> {
    using R = float2;
    __device__ static void get(R r, float (&x)[2]) {
        x[0] = r.x;
        x[1] = r.y;
    }
    __device__ static R put(const float (&x)[2]) { return make_float2(x[0], x[1]); }
};

// Rows [..][ld] of activations of one batch row, from channel c0 on; the row is the
// wave's, the channels behind it the lane's.
template <int ACT, int V> struct Rows {
    using L = Lane<ACT, V>;
    using R = typename L::R;
    using T = typename Act<ACT>::T;
    T *base;
    int64_t ld;
    uint32_t lane;
    __device__ Rows(const void *p, int64_t ld, int64_t first, int64_t c0, uint32_t lane)
        : base(const_cast<T *>(static_cast<const T *>(p)) + first * ld + c0), ld(ld), lane(lane) {}
    __device__ R load(int64_t t) const { return *reinterpret_cast<const R *>(base + t * ld + lane); }
    __device__ void store(int64_t t, const float (&x)[V]) const {
        *reinterpret_cast<R *>(base + t * ld + lane) = L::put(x);
    }
};

// ------------------------------------------------------------------ joining workgroups

// slots[place][channel], then ends[group][channel] of a row's tile; a counter before all.
struct Join {
    uint64_t *slots, *ends;
};

__device__ __forceinline__ uint64_t *counter_of(const RecurArgs &a) { return reinterpret_cast<uint64_t *>(a.ws); }

template <int V> __device__ __forceinline__ Join join_of(const RecurArgs &a, int64_t row_tile, int places) {
    const int groups = (places + kGroup - 1) / kGroup;
    uint64_t *p = reinterpret_cast<uint64_t *>(a.ws + 256) + row_tile * (places + groups) * (kWave * V);
    return {p, p + (int64_t)places * (kWave * V)};
}

__device__ __forceinline__ void put_word(uint64_t *p, float A, float H) {
    uint32_t bits = __float_as_uint(A);
    if (bits == 0xffffffffu) bits = 0x7fc00000u;  // no NaN may look like the mark
    __hip_atomic_store(p, (uint64_t)bits << 32 | __float_as_uint(H), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What comes into the workgroup at `place`, whose own run is (A, H) (a lane's
// channels); first: what comes into place 0.
template <int V>
__device__ __forceinline__ void join(const Join &j, int place, int places, const float (&A)[V], const float (&H)[V],
                                     const float (&first)[V], float (&in)[V]) {
    const int lane = threadIdx.x % kWave, group = place / kGroup, member = place % kGroup;
    const bool last = member == kGroup - 1;
    uint64_t *own = j.slots + ((int64_t)place * kWave + lane) * V, *end = j.ends + ((int64_t)group * kWave + lane) * V;
    if (place == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            in[e] = first[e];
            if (places > 1) put_word(own + e, 0.0f, fmaf(A[e], in[e], H[e]));
        }
        return;
    }
    if (!last) {
#pragma unroll
        for (int e = 0; e < V; ++e) put_word(own + e, A[e], H[e]);
    }
    // the group before, then this group's earlier members
    uint64_t words[kGroup][V];
    for (;;) {
        bool there = true;
#pragma unroll
        for (int k = 0; k < kGroup; ++k) {
            const uint64_t *p = k == 0 ? end - (int64_t)kWave * V : own - (int64_t)(member - k + 1) * kWave * V;
            if (k == 0 ? group > 0 : k - 1 < member) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    words[k][e] = __hip_atomic_load(p + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    there = there && words[k][e] != kMark;
                }
            }
        }
        if (__all(there)) break;
        __builtin_amdgcn_s_sleep(2);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        in[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
            if (k == 0 ? group > 0 : k - 1 < member)
                in[e] = fmaf(__uint_as_float((uint32_t)(words[k][e] >> 32)), in[e], __uint_as_float((uint32_t)words[k][e]));
        if (last) put_word(end + e, 0.0f, fmaf(A[e], in[e], H[e]));
    }
}

// The workgroup's number: drawn, where workgroups wait for each other.
__device__ __forceinline__ int64_t draw_number(const RecurArgs &a, int places) {
    if (places == 1) return blockIdx.x;
    __shared__ uint32_t number;
    if (threadIdx.x == 0) number = atomicAdd(reinterpret_cast<unsigned int *>(counter_of(a)), 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane((int)number);
}

__global__ __launch_bounds__(256) void recurrence_mark_kernel(ulonglong2 *p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    p[i] = i < 16 ? ulonglong2{0, 0} : ulonglong2{kMark, kMark};  // 256 bytes of counter before the words
}

// ------------------------------------------------------------------ a prompt

template <int ACT, int GATE, int INPUT, int V, int W, int T>
__global__ __launch_bounds__(W *kWave) void recurrence_kernel(RecurArgs a, int places) {
    using Lane = Lane<ACT, V>;
    using R = typename Lane::R;
    constexpr int kRun = W * T;
    __shared__ float2 runs[W][kWave * V];
    __shared__ float came[kWave * V];
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t tiles = (a.D + kWave * V - 1) / (kWave * V), number = draw_number(a, places);
    const int place = (int)(number / (a.B * tiles));
    const int64_t row_tile = number % (a.B * tiles), b = row_tile / tiles, c0 = row_tile % tiles * (kWave * V);
    const bool mine = c0 + lane * V < a.D;
    // lanes past the last channel read its neighbours' and write nothing
    const int64_t at = mine ? lane * V : a.D - V - c0;
    const int64_t n = row_length(a, b), t0 = (int64_t)place * kRun + w * T;
    const Rows<ACT, V> y(a.y, a.ld_y, b * a.L, c0, (uint32_t)(lane * V));
    const float zero[V] = {};
    if (place > 0 && (int64_t)place * kRun >= n) {
        for (int64_t t = t0; t < t0 + T && t < a.L; ++t)
            if (mine) y.store(t, zero);
        return;
    }
    float f[T][V], x[T][V];
    R q[T];
    if (n > 0) {
        // rows past the end: the last one again, not used
        const Rows<ACT, V> gr(a.g, a.ld_g, b * a.L, c0, (uint32_t)at), vr(a.v, a.ld_v, b * a.L, c0, (uint32_t)at);
        const Rows<ACT, V> qr(a.q ? a.q : a.g, a.q ? a.ld_q : a.ld_g, b * a.L, c0, (uint32_t)at);
        R g[T], v[T];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int64_t t = t0 + j < n ? t0 + j : n - 1;
            g[j] = gr.load(t);
            v[j] = vr.load(t);
        }
        if (a.q) {
#pragma unroll
            for (int j = 0; j < T; ++j) q[j] = qr.load(t0 + j < n ? t0 + j : n - 1);
        }
#pragma unroll
        for (int j = 0; j < T; ++j) {
            Lane::get(g[j], f[j]);
            Lane::get(v[j], x[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float i;
                gate_of<GATE, INPUT>(f[j][e], f[j][e], i);
                x[j][e] = t0 + j < n ? i * x[j][e] : 0.0f;
                f[j][e] = t0 + j < n ? f[j][e] : 1.0f;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f[j][e] = 1.0f;
                x[j][e] = 0.0f;
            }
    }
    float A[V], H[V], h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        A[e] = 1.0f;
        H[e] = 0.0f;
#pragma unroll
        for (int j = 0; j < T; ++j) {
            H[e] = fmaf(f[j][e], H[e], x[j][e]);
            A[e] *= f[j][e];
        }
    }
    // the state before everything (another lane's, past the last channel: not used)
    float first[V] = {};
    if (a.state_in && (W == 1 || w == W - 1) && place == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) first[e] = a.state_in[b * a.D + c0 + at + e];
    }
    if constexpr (W == 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = first[e];
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) runs[w][lane * V + e] = make_float2(A[e], H[e]);
        __syncthreads();
        float pA[V], pH[V];  // the waves before
#pragma unroll
        for (int e = 0; e < V; ++e) {
            pA[e] = 1.0f;
            pH[e] = 0.0f;
        }
        for (int k = 0; k < w; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 r = runs[k][lane * V + e];
                pH[e] = fmaf(r.x, pH[e], r.y);
                pA[e] *= r.x;
            }
        if (w == W - 1) {
            float in[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                H[e] = fmaf(A[e], pH[e], H[e]);
                A[e] *= pA[e];
                in[e] = first[e];
            }
            if (places > 1) join<V>(join_of<V>(a, row_tile, places), place, places, A, H, first, in);
#pragma unroll
            for (int e = 0; e < V; ++e) came[lane * V + e] = in[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = fmaf(pA[e], came[lane * V + e], pH[e]);
    }
    if (a.chunk_states && t0 % kRecurChunk == 0 && t0 < n && mine) {
        const int64_t chunks = (a.L + kRecurChunk - 1) / kRecurChunk;
        float *p = a.chunk_states + (b * chunks + t0 / kRecurChunk) * a.D + c0 + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) p[e] = h[e];
    }
#pragma unroll
    for (int j = 0; j < T; ++j) {
        float out[V];
        if (a.q && n > 0) Lane::get(q[j], out);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            h[e] = fmaf(f[j][e], h[e], x[j][e]);
            out[e] = t0 + j >= n ? 0.0f : a.q ? out[e] * h[e] : h[e];
        }
        if (t0 + j < a.L && mine) y.store(t0 + j, out);
    }
    // the row's last run: what is past its end left h as it was
    if (w == W - 1 && mine && (int64_t)(place + 1) * kRun >= n) {
#pragma unroll
        for (int e = 0; e < V; ++e) a.state_out[b * a.D + c0 + lane * V + e] = h[e];
    }
}

// ------------------------------------------------------------------ backward

template <int ACT, int GATE, int INPUT, int V, int W, int T>
__global__ __launch_bounds__(W *kWave) void recurrence_backward_kernel(RecurArgs a, int places) {
    using Lane = Lane<ACT, V>;
    using R = typename Lane::R;
    constexpr int kRun = W * T;
    static_assert(kRun <= kRecurChunk && kRecurChunk % kRun == 0, "a run starts from one kept state");
    __shared__ float4 runs[W][kWave * V];  // A, H, K
    __shared__ float came[kWave * V];
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t tiles = (a.D + kWave * V - 1) / (kWave * V), number = draw_number(a, places);
    const int run = places - 1 - (int)(number / (a.B * tiles));  // the last ones first
    const int64_t row_tile = number % (a.B * tiles), b = row_tile / tiles, c0 = row_tile % tiles * (kWave * V);
    const bool mine = c0 + lane * V < a.D;
    const int64_t at = mine ? lane * V : a.D - V - c0;
    const int64_t n = row_length(a, b), t0 = (int64_t)run * kRun + w * T;
    const Rows<ACT, V> dqr(a.dq, a.ld_dq, b * a.L, c0, (uint32_t)(lane * V));
    const Rows<ACT, V> dgr(a.dg, a.ld_dg, b * a.L, c0, (uint32_t)(lane * V));
    const Rows<ACT, V> dvr(a.dv, a.ld_dv, b * a.L, c0, (uint32_t)(lane * V));
    const float zero[V] = {};
    auto clear = [&](int64_t from) {
        for (int64_t t = from > t0 ? from : t0; t < t0 + T && t < a.L; ++t)
            if (mine) {
                if (a.q) dqr.store(t, zero);
                dgr.store(t, zero);
                dvr.store(t, zero);
            }
    };
    if (run > 0 && (int64_t)run * kRun >= n) {
        clear(t0);
        return;
    }
    const int last_run = n > 0 ? (int)((n - 1) / kRun) : 0;
    float back[V] = {};
    if (a.dstate_out && run == last_run) {
#pragma unroll
        for (int e = 0; e < V; ++e) back[e] = a.dstate_out[b * a.D + c0 + at + e];
    }
    if (n == 0) {
        clear(0);
        if (w == 0 && mine && a.dstate_in) {
#pragma unroll
            for (int e = 0; e < V; ++e) a.dstate_in[b * a.D + c0 + lane * V + e] = back[e];
        }
        return;
    }
    const Rows<ACT, V> gr(a.g, a.ld_g, b * a.L, c0, (uint32_t)at), vr(a.v, a.ld_v, b * a.L, c0, (uint32_t)at);
    const Rows<ACT, V> qr(a.q ? a.q : a.g, a.q ? a.ld_q : a.ld_g, b * a.L, c0, (uint32_t)at);
    const Rows<ACT, V> dyr(a.dy, a.ld_dy, b * a.L, c0, (uint32_t)at);
    R g[T], v[T], q[T], dy[T];
#pragma unroll
    for (int j = 0; j < T; ++j) {
        const int64_t t = t0 + j < n ? t0 + j : n - 1;
        g[j] = gr.load(t);
        v[j] = vr.load(t);
        dy[j] = dyr.load(t);
    }
    if (a.q) {
#pragma unroll
        for (int j = 0; j < T; ++j) q[j] = qr.load(t0 + j < n ? t0 + j : n - 1);
    }
    float h[V];
    {
        const int64_t chunks = (a.L + kRecurChunk - 1) / kRecurChunk;
        const float *p = a.chunk_states + (b * chunks + (int64_t)run * kRun / kRecurChunk) * a.D + c0 + at;
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = p[e];
    }
    float f[T][V], x[T][V], A[V], H[V], K[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        A[e] = 1.0f;
        H[e] = K[e] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < T; ++j) {
        Lane::get(g[j], f[j]);
        Lane::get(v[j], x[j]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float i;
            gate_of<GATE, INPUT>(f[j][e], f[j][e], i);
            x[j][e] = t0 + j < n ? i * x[j][e] : 0.0f;
            f[j][e] = t0 + j < n ? f[j][e] : 1.0f;
            H[e] = fmaf(f[j][e], H[e], x[j][e]);
            A[e] *= f[j][e];
        }
    }
    // q dy of a token, 0 past the end
    auto given = [&](int j, float (&s)[V]) {
        float d[V];
        Lane::get(dy[j], d);
        if (a.q) Lane::get(q[j], s);
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] = t0 + j >= n ? 0.0f : a.q ? s[e] * d[e] : d[e];
    };
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
        float s[V];
        given(j, s);
#pragma unroll
        for (int e = 0; e < V; ++e) K[e] = f[j][e] * (s[e] + K[e]);
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) runs[w][lane * V + e] = make_float4(A[e], H[e], K[e], 0.0f);
        __syncthreads();
        for (int k = 0; k < w; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float4 r = runs[k][lane * V + e];
                h[e] = fmaf(r.x, h[e], r.y);
            }
        float pA[V], pK[V];  // the waves behind
#pragma unroll
        for (int e = 0; e < V; ++e) {
            pA[e] = 1.0f;
            pK[e] = 0.0f;
        }
        for (int k = W - 1; k > w; --k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float4 r = runs[k][lane * V + e];
                pK[e] = fmaf(r.x, pK[e], r.z);
                pA[e] *= r.x;
            }
        if (w == 0) {
            float in[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                K[e] = fmaf(A[e], pK[e], K[e]);
                A[e] *= pA[e];
                in[e] = back[e];
            }
            if (places > 1) join<V>(join_of<V>(a, row_tile, places), last_run - run, last_run + 1, A, K, back, in);
#pragma unroll
            for (int e = 0; e < V; ++e) came[lane * V + e] = in[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) back[e] = fmaf(pA[e], came[lane * V + e], pK[e]);
    }
    // the h before every token, in x's place; dq on the way
#pragma unroll
    for (int j = 0; j < T; ++j) {
        float d[V];
        Lane::get(dy[j], d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float before = h[e];
            h[e] = fmaf(f[j][e], h[e], x[j][e]);
            x[j][e] = before;
            d[e] *= h[e];
        }
        if (a.q && t0 + j < n && mine) dqr.store(t0 + j, d);
    }
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
        float s[V], gj[V], vj[V], dg[V], dv[V];
        given(j, s);
        Lane::get(g[j], gj);
        Lane::get(v[j], vj);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float ff, i, df, di;
            gate_grad<GATE, INPUT>(gj[e], ff, i, df, di);
            const float dh = s[e] + back[e];
            dg[e] = dh * fmaf(df, x[j][e], di * vj[e]);
            dv[e] = dh * i;
            back[e] = f[j][e] * dh;
        }
        if (t0 + j < n && mine) {
            dgr.store(t0 + j, dg);
            dvr.store(t0 + j, dv);
        }
    }
    clear(n);
    if (run == 0 && w == 0 && mine && a.dstate_in) {
#pragma unroll
        for (int e = 0; e < V; ++e) a.dstate_in[b * a.D + c0 + lane * V + e] = back[e];
    }
}

// ------------------------------------------------------------------ one token

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

constexpr int kWaves = 8, kLong = 16, kShort = 8;  // waves, and tokens of a wave

// Tokens of a workgroup of a prompt: up to 8 in one wave, else 8 a wave to 64 in
// all, else 16 a wave.
int prompt_run(int64_t L) { return L <= kShort ? kShort : L <= kWaves * kShort ? kWaves * kShort : kWaves * kLong; }
int backward_run(int64_t L) { return L <= kShort ? kShort : kRecurChunk; }
int places_of(int64_t L, int run) { return L > 0 ? (int)((L + run - 1) / run) : 1; }

// Pairs of channels a lane where all rows have them aligned.
bool in_pairs(const RecurArgs &a) {
    const uintptr_t e = a.act == kBF16 ? 4 : 8;
    auto ok = [&](const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % e == 0 && (ld % 2 == 0 || a.L * a.B <= 1); };
    return a.D % 2 == 0 && ok(a.q, a.ld_q) && ok(a.g, a.ld_g) && ok(a.v, a.ld_v) && ok(a.y, a.ld_y) && ok(a.dy, a.ld_dy) &&
           ok(a.dq, a.ld_dq) && ok(a.dg, a.ld_dg) && ok(a.dv, a.ld_dv);
}

size_t words_bytes(int64_t B, int64_t D, int places) {
    const int64_t channels = (D + 2 * kWave - 1) / (2 * kWave) * (2 * kWave), groups = (places + kGroup - 1) / kGroup;
    return places > 1 ? 256 + (size_t)(B * channels) * (size_t)(places + groups) * sizeof(uint64_t) : 0;
}

hipError_t mark_words(const RecurArgs &a, int places, hipStream_t stream) {
    const int64_t n = (int64_t)(words_bytes(a.B, a.D, places) / sizeof(ulonglong2));
    if (n > 0) recurrence_mark_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, stream>>>(reinterpret_cast<ulonglong2 *>(a.ws), n);
    return hipGetLastError();
}

}  // namespace

size_t recurrence_workspace(int64_t B, int64_t D, int64_t L) {
    const size_t p = words_bytes(B, D, places_of(L, prompt_run(L))), q = words_bytes(B, D, places_of(L, backward_run(L)));
    return p > q ? p : q;
}

hipError_t launch_recurrence_prefill(const RecurArgs &a, hipStream_t stream) {
    const int run = prompt_run(a.L), places = places_of(a.L, run);
    const hipError_t e = mark_words(a, places, stream);
    if (e != hipSuccess) return e;
    return for_types(a, [&](auto act, auto gate, auto input) {
        constexpr int C = decltype(act)::value, G = decltype(gate)::value, I = decltype(input)::value;
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            const dim3 grid((unsigned)(a.B * ((a.D + kWave * V - 1) / (kWave * V)) * places));
            if (run == kShort) recurrence_kernel<C, G, I, V, 1, kShort><<<grid, kWave, 0, stream>>>(a, places);
            else if (run == kWaves * kShort) recurrence_kernel<C, G, I, V, kWaves, kShort><<<grid, kWaves * kWave, 0, stream>>>(a, places);
            else recurrence_kernel<C, G, I, V, kWaves, kLong><<<grid, kWaves * kWave, 0, stream>>>(a, places);
        };
        if (in_pairs(a)) go(std::integral_constant<int, 2>{});
        else go(std::integral_constant<int, 1>{});
    });
}

hipError_t launch_recurrence_backward(const RecurArgs &a, hipStream_t stream) {
    const int run = backward_run(a.L), places = places_of(a.L, run);
    const hipError_t e = mark_words(a, places, stream);
    if (e != hipSuccess) return e;
    return for_types(a, [&](auto act, auto gate, auto input) {
        constexpr int C = decltype(act)::value, G = decltype(gate)::value, I = decltype(input)::value;
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            const dim3 grid((unsigned)(a.B * ((a.D + kWave * V - 1) / (kWave * V)) * places));
            if (run == kShort) recurrence_backward_kernel<C, G, I, V, 1, kShort><<<grid, kWave, 0, stream>>>(a, places);
            else recurrence_backward_kernel<C, G, I, V, kWaves, kShort><<<grid, kWaves * kWave, 0, stream>>>(a, places);
        };
        if (in_pairs(a)) go(std::integral_constant<int, 2>{});
        else go(std::integral_constant<int, 1>{});
    });
}

hipError_t launch_recurrence_decode(const RecurArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * ((a.D + 255) / 256)));
    return for_types(a, [&](auto act, auto gate, auto input) {
        recurrence_token_kernel<decltype(act)::value, decltype(gate)::value, decltype(input)::value><<<grid, 256, 0, stream>>>(a);
    });
}

}  // namespace hm
