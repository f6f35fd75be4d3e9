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
// Workgroups join through words of the workspace, (A, H) as one of 64 bits a channel,
// filled with a mark beforehand; a word that is not the mark is there.  A workgroup
// waits for its group's earlier ones and for the h behind the group before.  Which
// words, and the order of the products, are fixed by its place, so results do not
// depend on timing.  Places go by a counter that each workgroup draws from when it
// starts, earlier runs first: whom it waits for has started, and needs nothing from
// later ones, so every wait ends.
//
// What bounds it (MI355X): HBM.  65536 x 4096 bfloat16 tokens, 2.15 GB: 420 us, 5.1
// TB/s, as a large copy; without the join 379.  A workgroup's 8 waves hold 128 tokens of
// 128 channels, two workgroups a CU (at most 128 registers: a third of a wave more and
// there is one, which waits for others with nothing else to do: 539 us).  Runs of 64
// tokens: 558 us, more to draw, mark and join for the same bytes.  Joined one by one in
// groups of 8, the chain of places 8 times as long and waited for after the words: 586.
#include "hm_internal.hpp"

namespace hm {
namespace {

constexpr int kGroup = 8;          // workgroups that join one by one
constexpr uint64_t kMark = ~0ull;  // a word that is not there yet
constexpr int kPatience = 1 << 20; // looks at a word

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

constexpr int kStream = 2;  // aux of the buffer builtins: non-temporal

// Memory of a lane's V neighbouring channels of a token, and its values.  Results are
// stored past the caches, where the inputs are more use (8 x 2048 x 2048 bfloat16,
// forward and backward: 159 us against 179).
template <int BYTES> struct Piece;
template <> struct Piece<2> {
    using R = uint16_t;
    template <bool ONCE> __device__ static R load(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t row) {
        return __builtin_amdgcn_raw_buffer_load_b16(r, at, row, ONCE ? kStream : 0);
    }
    __device__ static void store(R x, __amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t row) {
        __builtin_amdgcn_raw_buffer_store_b16(x, r, at, row, kStream);
    }
};
template <> struct Piece<4> {
    using R = uint32_t;
    template <bool ONCE> __device__ static R load(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t row) {
        return __builtin_amdgcn_raw_buffer_load_b32(r, at, row, ONCE ? kStream : 0);
    }
    __device__ static void store(R x, __amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t row) {
        __builtin_amdgcn_raw_buffer_store_b32(x, r, at, row, kStream);
    }
};
template <int ACT, int V> struct Lane : Piece<V * Act<ACT>::kBytes> {
    using R = typename Piece<V * Act<ACT>::kBytes>::R;
    __device__ static void get(R r, float (&x)[V]) {
        if constexpr (ACT == kF32) {
            x[0] = __uint_as_float(r);
        } else {
            x[0] = bf16_lo(r);
            if constexpr (V == 2) x[1] = bf16_hi(r);
        }
    }
    __device__ static R put(const float (&x)[V]) {
        if constexpr (ACT == kF32) return __float_as_uint(x[0]);
        else if constexpr (V == 1) return (uint16_t)f32_to_bf16(x[0]);
        else return pack_bf16x2(x[0], x[1]);
    }
};

// A tile's first channel.  The last tile of an odd number of channels in pairs begins one
// earlier: that channel's results come from two workgroups, and are the same.
template <int V> __device__ __forceinline__ int64_t tile_begin(uint32_t tile, uint32_t tiles, int64_t D) {
    return (int64_t)tile * (kWave * V) - (tile + 1 == tiles ? D % V : 0);
}

// Hides from the compiler that x is what it was.
template <typename R> __device__ __forceinline__ void opaque(R &x) { asm volatile("" : "+v"(x)); }

// `rows` rows of activations of a tile of channels from row `first` on, none where
// there is no memory: what lies behind the last one reads as 0 and is not written, nor
// is a lane past the last channel.  Offsets stay below 2^31, by kRecurRows and
// kRecurMostStride.
constexpr uint32_t kNowhere = 0x80000000u;
template <int ACT, int V> struct Rows {
    using L = Lane<ACT, V>;
    using R = typename L::R;
    static constexpr uint32_t kBytes = Act<ACT>::kBytes;
    __amdgpu_buffer_rsrc_t region;
    uint32_t at, step;
    __device__ Rows(const void *p, int64_t ld, int64_t first, int64_t rows, int64_t c0, int64_t D, int lane) {
        const int64_t width = D - c0 < kWave * V ? D - c0 : kWave * V;
        const bool any = p && rows > 0;
        region = make_region(static_cast<const typename Act<ACT>::T *>(p) + (any ? first * ld + c0 : 0),
                             any ? (uint32_t)((rows - 1) * ld + width) * kBytes : 0u);
        step = (uint32_t)(ld < kRecurMostStride ? ld : kRecurMostStride) * kBytes;  // (larger ones come with one row)
        at = lane * V < width ? lane * V * kBytes : kNowhere;
    }
    // ALL: every row is there, and its offset need not count for the bounds
    template <bool ALL, bool ONCE> __device__ R load(int j) const {
        return ALL ? L::template load<ONCE>(region, at, j * step) : L::template load<ONCE>(region, at + j * step, 0);
    }
    template <bool ALL> __device__ void store(int j, const float (&x)[V]) const {
        ALL ? L::store(L::put(x), region, at, j * step) : L::store(L::put(x), region, at + j * step, 0);
    }
};

// ------------------------------------------------------------------ joining workgroups

// The workspace: a counter for each row's tile of channels, 128 bytes apart, then its
// words: (A, H) of each place, (A, H) of each group of kGroup places, and the h behind
// each kGroup groups, a word a channel each.
constexpr int kCounter = 128;

__host__ __device__ constexpr int groups_of(int n) { return (n + kGroup - 1) / kGroup; }
__host__ __device__ constexpr int64_t words_of(int places) {
    return (int64_t)places + groups_of(places) + groups_of(groups_of(places));
}

__device__ __forceinline__ void put_word(uint64_t *p, float A, float H) {
    uint32_t bits = __float_as_uint(A);
    if (bits == 0xffffffffu) bits = 0x7fc00000u;  // no NaN may look like the mark
    __hip_atomic_store(p, (uint64_t)bits << 32 | __float_as_uint(H), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A lane's V words at p, as soon as they are there.  (A word that never comes, in a
// workspace that another call writes to at the same time, is taken as the mark, a NaN,
// after about a second.)
template <int V> __device__ __forceinline__ void wait_words(const uint64_t *p, float2 *out) {
    uint64_t word[V];
    for (int turn = 0; turn < kPatience; ++turn) {
        bool there = true;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            word[e] = __hip_atomic_load(p + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            there = there && word[e] != kMark;
        }
        if (__all(there)) break;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        out[e] = make_float2(__uint_as_float((uint32_t)(word[e] >> 32)), __uint_as_float((uint32_t)word[e]));
}

template <int V> struct JoinShared {
    float2 members[kGroup - 1][kWave * V], groups[kGroup - 1][kWave * V], before[kWave * V];
};

// What comes into the workgroup at `place` (a lane's channels).  Its last wave has its
// own run (A, H); first: what comes into place 0.  Every wave looks out for other words:
// those of the places before it in its group, of the groups before that in their group,
// and the h before those, which is the only chain: one link for kGroup^2 places.
template <int V, int W>
__device__ __forceinline__ void join(const RecurArgs &a, uint32_t row_tile, uint32_t row_tiles, int places, int place, int w,
                                     const float (&A)[V], const float (&H)[V], const float (&first)[V], JoinShared<V> &sh,
                                     float (&in)[V]) {
    const int lane = threadIdx.x % kWave, at = lane * V;
    uint64_t *slots = reinterpret_cast<uint64_t *>(a.ws + (int64_t)row_tiles * kCounter) +
                      (int64_t)row_tile * words_of(places) * (kWave * V) + at;
    uint64_t *groups = slots + (int64_t)places * (kWave * V);
    uint64_t *ends = groups + (int64_t)groups_of(places) * (kWave * V);
    const int group = place / kGroup, member = place % kGroup, end = group / kGroup, behind = group % kGroup;
    auto word = [&](uint64_t *p, int k) { return p + (int64_t)k * (kWave * V); };
    if (w == W - 1 && member < kGroup - 1) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            put_word(word(slots, place) + e, place == 0 ? 0.0f : A[e], place == 0 ? fmaf(A[e], first[e], H[e]) : H[e]);
    }
    if (place == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) in[e] = first[e];
        return;
    }
    for (int k = w; k < member; k += W) wait_words<V>(word(slots, group * kGroup + k), &sh.members[k][at]);
    if (member == kGroup - 1 && behind < kGroup - 1) {  // the whole group's, before waiting for others
        __syncthreads();
        if (w == W - 1) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float gA = 1.0f, gH = 0.0f;
#pragma unroll
                for (int k = 0; k < kGroup - 1; ++k) {
                    const float2 m = sh.members[k][at + e];
                    gH = fmaf(m.x, gH, m.y);
                    gA *= m.x;
                }
                put_word(word(groups, group) + e, gA * A[e], fmaf(A[e], gH, H[e]));
            }
        }
    }
    for (int k = w; k < behind; k += W) wait_words<V>(word(groups, end * kGroup + k), &sh.groups[k][at]);
    if (end > 0 && w == W - 1) wait_words<V>(word(ends, end - 1), &sh.before[at]);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) {
        in[e] = end > 0 ? sh.before[at + e].y : 0.0f;
        for (int k = 0; k < behind; ++k) in[e] = fmaf(sh.groups[k][at + e].x, in[e], sh.groups[k][at + e].y);
        for (int k = 0; k < member; ++k) in[e] = fmaf(sh.members[k][at + e].x, in[e], sh.members[k][at + e].y);
    }
    if (w == W - 1 && member == kGroup - 1 && behind == kGroup - 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) put_word(word(ends, end) + e, 0.0f, fmaf(A[e], in[e], H[e]));
    }
}

// The workgroup's place in its row's tile: drawn, where workgroups wait for each other.
// (One counter for all was drawn from every 14 ns at most: 65536 x 4096 tokens in runs
// of 64, 460 us of drawing.)
__device__ __forceinline__ int draw_place(const RecurArgs &a, uint32_t row_tile, int places) {
    if (places == 1) return 0;
    __shared__ uint32_t place;
    if (threadIdx.x == 0) place = atomicAdd(reinterpret_cast<unsigned int *>(a.ws + (int64_t)row_tile * kCounter), 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane((int)place);
}

__global__ __launch_bounds__(256) void recurrence_mark_kernel(ulonglong2 *p, int64_t counters, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = i < counters ? ulonglong2{0, 0} : ulonglong2{kMark, kMark};
}

// ------------------------------------------------------------------ a prompt

template <int ACT, int GATE, int INPUT, int V, int W, int T, bool ONCE>
__global__ __launch_bounds__(W *kWave, 4) void recurrence_kernel(RecurArgs a, int places) {
    using Lane = Lane<ACT, V>;
    using R = typename Lane::R;
    constexpr int kRun = W * T;
    __shared__ float2 runs[W][kWave * V];
    __shared__ JoinShared<V> joined;
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t tiles = (uint32_t)((a.D + kWave * V - 1) / (kWave * V)), row_tiles = (uint32_t)a.B * tiles;
    const uint32_t row_tile = blockIdx.x % row_tiles, tile = row_tile % tiles;
    const int place = draw_place(a, row_tile, places);
    if (place >= places) return;  // (no counter of this call's says so)
    const int64_t b = row_tile / tiles, c0 = tile_begin<V>(tile, tiles, a.D);
    const bool mine = c0 + lane * V < a.D;
    // lanes past the last channel read their neighbours' states and write nothing
    const int64_t at = mine ? lane * V : a.D - V - c0;
    const int64_t n = row_length(a, b), r0 = (int64_t)place * kRun, t0 = r0 + w * T, first_row = b * a.L + t0;
    const Rows<ACT, V> y(a.y, a.ld_y, first_row, a.L - t0 < T ? a.L - t0 : T, c0, a.D, lane);
    if (place > 0 && r0 >= n) {
        const float zero[V] = {};
#pragma unroll
        for (int j = 0; j < T; ++j) y.template store<false>(j, zero);
        return;
    }
    const int64_t rows = n - t0 < T ? n - t0 : T;
    const Rows<ACT, V> gr(a.g, a.ld_g, first_row, rows, c0, a.D, lane);
    const Rows<ACT, V> vr(a.v, a.ld_v, first_row, rows, c0, a.D, lane);
    const Rows<ACT, V> qr(a.q, a.ld_q, first_row, rows, c0, a.D, lane);
    // whole: every token of the workgroup is before the row's end
    auto go = [&](auto whole) {
        constexpr bool ALL = decltype(whole)::value;
        R g[T], v[T], q[T];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            g[j] = gr.template load<ALL, ONCE>(j);
            v[j] = vr.template load<ALL, ONCE>(j);
        }
#pragma unroll
        for (int j = 0; j < T; ++j) q[j] = qr.template load<ALL, ONCE>(j);
        const int live = ALL ? T : rows > 0 ? (int)rows : 0;
        float f[T][V], x[T][V];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            Lane::get(g[j], f[j]);
            Lane::get(v[j], x[j]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float i;
                gate_of<GATE, INPUT>(f[j][e], f[j][e], i);
                x[j][e] = ALL || j < live ? i * x[j][e] : 0.0f;
                f[j][e] = ALL || j < live ? f[j][e] : 1.0f;
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
        if (a.state_in && place == 0) {
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
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    H[e] = fmaf(A[e], pH[e], H[e]);
                    A[e] *= pA[e];
                }
            }
            if (places > 1) {
                join<V, W>(a, row_tile, row_tiles, places, place, w, A, H, first, joined, h);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) h[e] = first[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) h[e] = fmaf(pA[e], h[e], pH[e]);
        }
        if (a.chunk_states && t0 % kRecurChunk == 0 && live > 0 && mine) {
            const int64_t chunks = (a.L + kRecurChunk - 1) / kRecurChunk;
            float *p = a.chunk_states + (b * chunks + t0 / kRecurChunk) * a.D + c0 + lane * V;
#pragma unroll
            for (int e = 0; e < V; ++e) p[e] = h[e];
        }
#pragma unroll
        for (int j = 0; j < T; ++j) {
            float out[V];
            Lane::get(q[j], out);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[e] = fmaf(f[j][e], h[e], x[j][e]);
                out[e] = !ALL && j >= live ? 0.0f : a.q ? out[e] * h[e] : h[e];
            }
            y.template store<ALL>(j, out);
        }
        // the row's last run: what is past its end left h as it was
        if (w == W - 1 && mine && r0 + kRun >= n) {
#pragma unroll
            for (int e = 0; e < V; ++e) a.state_out[b * a.D + c0 + lane * V + e] = h[e];
        }
    };
    if (n - r0 >= kRun) go(std::true_type{});
    else go(std::false_type{});
}

// ------------------------------------------------------------------ backward

template <int ACT, int GATE, int INPUT, int V, int W, int T, bool ONCE>
__global__ __launch_bounds__(W *kWave, 4) void recurrence_backward_kernel(RecurArgs a, int places) {
    using Lane = Lane<ACT, V>;
    using R = typename Lane::R;
    constexpr int kRun = W * T;
    static_assert(kRun <= kRecurChunk && kRecurChunk % kRun == 0, "a run starts from one kept state");
    __shared__ float4 runs[W][kWave * V];  // A, H, K
    __shared__ JoinShared<V> joined;
    const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t tiles = (uint32_t)((a.D + kWave * V - 1) / (kWave * V)), row_tiles = (uint32_t)a.B * tiles;
    const uint32_t row_tile = blockIdx.x % row_tiles, tile = row_tile % tiles;
    const int run = places - 1 - draw_place(a, row_tile, places);  // the last ones first
    if (run < 0) return;
    const int64_t b = row_tile / tiles, c0 = tile_begin<V>(tile, tiles, a.D);
    const bool mine = c0 + lane * V < a.D;
    const int64_t at = mine ? lane * V : a.D - V - c0;
    const int64_t n = row_length(a, b), r0 = (int64_t)run * kRun, t0 = r0 + w * T, first_row = b * a.L + t0;
    const int64_t all = a.L - t0 < T ? a.L - t0 : T;
    const Rows<ACT, V> dqr(a.dq, a.ld_dq, first_row, all, c0, a.D, lane);
    const Rows<ACT, V> dgr(a.dg, a.ld_dg, first_row, all, c0, a.D, lane);
    const Rows<ACT, V> dvr(a.dv, a.ld_dv, first_row, all, c0, a.D, lane);
    if (r0 >= n) {  // behind the row's end, or a row of none
        const float zero[V] = {};
#pragma unroll
        for (int j = 0; j < T; ++j) {
            dqr.template store<false>(j, zero);
            dgr.template store<false>(j, zero);
            dvr.template store<false>(j, zero);
        }
        if (run == 0 && w == 0 && mine && a.dstate_in) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                a.dstate_in[b * a.D + c0 + lane * V + e] = a.dstate_out ? a.dstate_out[b * a.D + c0 + lane * V + e] : 0.0f;
        }
        return;
    }
    const int last_run = (int)((n - 1) / kRun);
    float back[V] = {};
    if (a.dstate_out && run == last_run) {
#pragma unroll
        for (int e = 0; e < V; ++e) back[e] = a.dstate_out[b * a.D + c0 + at + e];
    }
    const int64_t rows = n - t0 < T ? n - t0 : T;
    const Rows<ACT, V> gr(a.g, a.ld_g, first_row, rows, c0, a.D, lane);
    const Rows<ACT, V> vr(a.v, a.ld_v, first_row, rows, c0, a.D, lane);
    const Rows<ACT, V> qr(a.q, a.ld_q, first_row, rows, c0, a.D, lane);
    const Rows<ACT, V> dyr(a.dy, a.ld_dy, first_row, rows, c0, a.D, lane);
    auto go = [&](auto whole) {
        constexpr bool ALL = decltype(whole)::value;
        R g[T], v[T], q[T], dy[T];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            g[j] = gr.template load<ALL, ONCE>(j);
            v[j] = vr.template load<ALL, ONCE>(j);
        }
#pragma unroll
        for (int j = 0; j < T; ++j) {
            dy[j] = dyr.template load<ALL, ONCE>(j);
            q[j] = qr.template load<ALL, ONCE>(j);
        }
        const int live = ALL ? T : rows > 0 ? (int)rows : 0;
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
                x[j][e] = ALL || j < live ? i * x[j][e] : 0.0f;
                f[j][e] = ALL || j < live ? f[j][e] : 1.0f;
                H[e] = fmaf(f[j][e], H[e], x[j][e]);
                A[e] *= f[j][e];
            }
        }
        // q dy of a token, 0 past the end
        auto given = [&](int j, float (&s)[V]) {
            float d[V];
            Lane::get(dy[j], d);
            Lane::get(q[j], s);
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] = !ALL && j >= live ? 0.0f : a.q ? s[e] * d[e] : d[e];
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
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    K[e] = fmaf(A[e], pK[e], K[e]);
                    A[e] *= pA[e];
                }
            }
            if (last_run > 0) {
                float in[V];
                join<V, W>(a, row_tile, row_tiles, places, last_run - run, W - 1 - w, A, K, back, joined, in);
#pragma unroll
                for (int e = 0; e < V; ++e) back[e] = in[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) back[e] = fmaf(pA[e], back[e], pK[e]);
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
                d[e] = ALL || j < live ? d[e] * h[e] : 0.0f;
            }
            dqr.template store<ALL>(j, d);
        }
#pragma unroll
        for (int j = T - 1; j >= 0; --j) {
            float s[V], gj[V], vj[V], dg[V], dv[V];
            // the gate is formed again: kept, it would take the registers of a second workgroup
            opaque(g[j]);
            given(j, s);
            Lane::get(g[j], gj);
            Lane::get(v[j], vj);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float ff, i, df, di;
                gate_grad<GATE, INPUT>(gj[e], ff, i, df, di);
                const float dh = s[e] + back[e];
                dg[e] = ALL || j < live ? dh * fmaf(df, x[j][e], di * vj[e]) : 0.0f;
                dv[e] = ALL || j < live ? dh * i : 0.0f;
                back[e] = ALL || j < live ? ff * dh : dh;
            }
            dgr.template store<ALL>(j, dg);
            dvr.template store<ALL>(j, dv);
        }
        if (run == 0 && w == 0 && mine && a.dstate_in) {
#pragma unroll
            for (int e = 0; e < V; ++e) a.dstate_in[b * a.D + c0 + lane * V + e] = back[e];
        }
    };
    if (n - r0 >= kRun) go(std::true_type{});
    else go(std::false_type{});
}

// ------------------------------------------------------------------ one token

// V neighbouring channels a lane: 4 where rows and states are aligned for it (256 rows of
// 4096 bfloat16 channels through parents' states: 5.1 us, 6.9 with one), else one.
template <int ACT, int GATE, int INPUT, int V>
__global__ __launch_bounds__(256) void recurrence_token_kernel(RecurArgs a) {
    using A = Act<ACT>;
    using T = typename A::T;
    struct alignas(V * sizeof(T)) Values { T x[V]; };
    struct alignas(V * 4) States { float h[V]; };
    const int64_t tiles = (a.D + 256 * V - 1) / (256 * V), b = blockIdx.x / tiles;
    const int64_t c = blockIdx.x % tiles * (256 * V) + threadIdx.x * V;
    if (c >= a.D) return;
    int64_t from = b;
    if (a.src_rows) {
        const int64_t r = a.src_rows[b];
        if (r >= 0 && r < a.B) from = r;
    }
    const Values g = *reinterpret_cast<const Values *>(static_cast<const T *>(a.g) + b * a.ld_g + c);
    const Values v = *reinterpret_cast<const Values *>(static_cast<const T *>(a.v) + b * a.ld_v + c);
    Values q{}, y;
    if (a.q) q = *reinterpret_cast<const Values *>(static_cast<const T *>(a.q) + b * a.ld_q + c);
    States s = *reinterpret_cast<const States *>(a.state_in + from * a.D + c);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float f, i;
        gate_of<GATE, INPUT>(A::ld(&g.x[e]), f, i);
        s.h[e] = fmaf(f, s.h[e], i * A::ld(&v.x[e]));
        A::st(&y.x[e], a.q ? s.h[e] * A::ld(&q.x[e]) : s.h[e]);
    }
    *reinterpret_cast<States *>(a.state_out + b * a.D + c) = s;
    *reinterpret_cast<Values *>(static_cast<T *>(a.y) + b * a.ld_y + c) = y;
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
static_assert(kLong <= kRecurRows && kShort <= kRecurRows, "rows of a wave");

// Tokens of a workgroup.  A prompt: up to 8 in one wave, else 8 a wave where 64 are
// enough, else 16.  Backward 8 a wave, whose registers hold twice as much a token.
int prompt_run(int64_t L) { return L <= kShort ? kShort : L <= kWaves * kShort ? kWaves * kShort : kWaves * kLong; }
int backward_run(int64_t L) { return L <= kShort ? kShort : kWaves * kShort; }
int places_of(int64_t L, int run) { return L > 0 ? (int)((L + run - 1) / run) : 1; }

// Whether `tensors` inputs are read past the caches: non-temporal where they do not fit
// the 256 MB of Infinity Cache (65536 x 4096 bfloat16 tokens: 420 us against 454;
// backward over 8 x 2048 x 2048: 5 us of 80 less), else not, since backward finds there
// what the prompt has read (6 x 1501 x 1000 float32: 77 us for both against 99).
bool read_once(const RecurArgs &a, int tensors) {
    return a.B * a.L * a.D * (a.act == kBF16 ? 2 : 4) * (tensors - (a.q ? 0 : 1)) >= (int64_t(256) << 20);
}

// Pairs of bfloat16 channels a lane (4 bytes, as one float32 channel), aligned or not:
// 65536 x 4095 tokens 602 us against 841 with one, 8 x 2048 x 2047 63 and 79 with inputs
// in the caches (from HBM 74), backward 128 and 174; 9 x 7095 x 131, two tiles instead of
// three, 33 and 31.  An odd number only where there is a tile before the last one, and its
// states (or their gradients) are not replaced before the last tile has read the channel
// that both have.
bool in_pairs(const RecurArgs &a, const float *from, const float *to) {
    return a.act == kBF16 && (a.D % 2 == 0 || (a.D > 2 * kWave && (from != to || !to)));
}

size_t counters_bytes(int64_t B, int64_t D) { return (size_t)(B * ((D + kWave - 1) / kWave)) * kCounter; }

// (row tiles of 64 channels have the most counters, of more channels the most words)
size_t words_bytes(int64_t B, int64_t D, int places) {
    constexpr int64_t kTile = 2 * kWave;
    const int64_t channels = (D + kTile - 1) / kTile * kTile;
    return places > 1 ? counters_bytes(B, D) + (size_t)(B * channels * words_of(places)) * sizeof(uint64_t) : 0;
}

hipError_t mark_words(const RecurArgs &a, int V, int places, hipStream_t stream) {
    if (places == 1) return hipSuccess;
    const int64_t row_tiles = a.B * ((a.D + kWave * V - 1) / (kWave * V));
    const int64_t counters = row_tiles * (kCounter / 16), n = counters + row_tiles * words_of(places) * (kWave * V / 2);
    recurrence_mark_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, stream>>>(reinterpret_cast<ulonglong2 *>(a.ws), counters, n);
    return hipGetLastError();
}

}  // namespace

size_t recurrence_workspace(int64_t B, int64_t D, int64_t L) {
    const size_t p = words_bytes(B, D, places_of(L, prompt_run(L))), q = words_bytes(B, D, places_of(L, backward_run(L)));
    return p > q ? p : q;
}

hipError_t launch_recurrence_prefill(const RecurArgs &a, hipStream_t stream) {
    const int run = prompt_run(a.L), places = places_of(a.L, run);
    const int V = in_pairs(a, a.state_in, a.state_out) ? 2 : 1;
    const hipError_t e = mark_words(a, V, places, stream);
    if (e != hipSuccess) return e;
    const bool once = read_once(a, 3);
    return for_types(a, [&](auto act, auto gate, auto input) {
        constexpr int C = decltype(act)::value, G = decltype(gate)::value, I = decltype(input)::value;
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            const dim3 grid((unsigned)(a.B * ((a.D + kWave * V - 1) / (kWave * V)) * places));
            if (run == kShort) recurrence_kernel<C, G, I, V, 1, kShort, false><<<grid, kWave, 0, stream>>>(a, places);
            else if (run == kWaves * kShort) recurrence_kernel<C, G, I, V, kWaves, kShort, false><<<grid, kWaves * kWave, 0, stream>>>(a, places);
            else if (once) recurrence_kernel<C, G, I, V, kWaves, kLong, true><<<grid, kWaves * kWave, 0, stream>>>(a, places);
            else recurrence_kernel<C, G, I, V, kWaves, kLong, false><<<grid, kWaves * kWave, 0, stream>>>(a, places);
        };
        if constexpr (C == kBF16) {
            if (V > 1) return go(std::integral_constant<int, 2>{});
        }
        go(std::integral_constant<int, 1>{});
    });
}

hipError_t launch_recurrence_backward(const RecurArgs &a, hipStream_t stream) {
    const int run = backward_run(a.L), places = places_of(a.L, run);
    const int V = in_pairs(a, a.dstate_out, a.dstate_in) ? 2 : 1;
    const hipError_t e = mark_words(a, V, places, stream);
    if (e != hipSuccess) return e;
    const bool once = read_once(a, 4);
    return for_types(a, [&](auto act, auto gate, auto input) {
        constexpr int C = decltype(act)::value, G = decltype(gate)::value, I = decltype(input)::value;
        auto go = [&](auto v) {
            constexpr int V = decltype(v)::value;
            const dim3 grid((unsigned)(a.B * ((a.D + kWave * V - 1) / (kWave * V)) * places));
            if (run == kShort) recurrence_backward_kernel<C, G, I, V, 1, kShort, false><<<grid, kWave, 0, stream>>>(a, places);
            else if (once) recurrence_backward_kernel<C, G, I, V, kWaves, kShort, true><<<grid, kWaves * kWave, 0, stream>>>(a, places);
            else recurrence_backward_kernel<C, G, I, V, kWaves, kShort, false><<<grid, kWaves * kWave, 0, stream>>>(a, places);
        };
        if constexpr (C == kBF16) {
            if (V > 1) return go(std::integral_constant<int, 2>{});
        }
        go(std::integral_constant<int, 1>{});
    });
}

hipError_t launch_recurrence_decode(const RecurArgs &a, hipStream_t stream) {
    const uintptr_t e = a.act == kBF16 ? 8 : 16;
    auto ok = [&](const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % e == 0 && (ld % 4 == 0 || a.B == 1); };
    const bool four = a.D % 4 == 0 && ok(a.q, a.ld_q) && ok(a.g, a.ld_g) && ok(a.v, a.ld_v) && ok(a.y, a.ld_y) &&
                      reinterpret_cast<uintptr_t>(a.state_in) % 16 == 0 && reinterpret_cast<uintptr_t>(a.state_out) % 16 == 0;
    return for_types(a, [&](auto act, auto gate, auto input) {
        constexpr int C = decltype(act)::value, G = decltype(gate)::value, I = decltype(input)::value;
        if (four) recurrence_token_kernel<C, G, I, 4><<<dim3((unsigned)(a.B * ((a.D + 1023) / 1024))), 256, 0, stream>>>(a);
        else recurrence_token_kernel<C, G, I, 1><<<dim3((unsigned)(a.B * ((a.D + 255) / 256))), 256, 0, stream>>>(a);
    });
}

}  // namespace hm
