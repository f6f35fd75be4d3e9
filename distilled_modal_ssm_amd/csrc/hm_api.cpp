// hm_api.cpp -- the C ABI declared in include/hyena_modal.h.
//
// Every entry point validates its arguments on the host first (sizes, pointers,
// alignment, workspace) and returns a status without touching the GPU when they
// are wrong.  Valid calls build an argument block and enqueue kernels on the
// caller's stream; nothing here allocates, frees or synchronises.
#include "hyena_modal.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <mutex>

#include "hm_internal.hpp"

// Device scratch of hyena_modal_prefill_noalloc: the prefill workspace for
// callers that cannot allocate.  Each GPU the library runs on holds its own
// copy of this array (HM_NOALLOC_SCRATCH_BYTES) from module load until the
// process ends.  Host code never passes its name to a kernel: the name is a
// host-side stand-in, and the device address comes from hipGetSymbolAddress.
static __device__ __align__(256) unsigned char scratch[HM_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices] = {};

// The address of `scratch` on the current device, looked up once per device
// (with that device current) and kept.  No allocation happens here.
hm_status scratch_for_current_device(void **out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return HM_ERR_HIP;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *ptr = nullptr;
        if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) return HM_ERR_HIP;
        g_scratch_ptr[dev] = ptr;
    }
    *out = g_scratch_ptr[dev];
    return HM_OK;
}

constexpr int64_t kMaxElems = int64_t(1) << 46;  // guard against int64 overflow in offsets

bool aligned(const void *p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) % m) == 0; }

hm_status check_desc(const hm_desc *desc) {
    if (!desc) return HM_ERR_INVALID_ARG;
    if (desc->abi_version != HM_ABI_VERSION) return HM_ERR_INVALID_ARG;
    if (desc->act_dtype != HM_F32 && desc->act_dtype != HM_BF16) return HM_ERR_UNSUPPORTED;
    if (desc->batch < 0 || desc->channels < 1 || desc->heads < 1 || desc->modes < 1)
        return HM_ERR_INVALID_ARG;
    if (desc->channels % desc->heads != 0) return HM_ERR_INVALID_ARG;
    if (desc->modes > HM_MAX_MODES) return HM_ERR_UNSUPPORTED;
    if (!desc->poles || !desc->residues || !desc->skip) return HM_ERR_INVALID_ARG;
    if (!aligned(desc->poles, 8) || !aligned(desc->residues, 8) || !aligned(desc->skip, 4))
        return HM_ERR_UNSUPPORTED;
    if (desc->batch > kMaxElems / desc->channels) return HM_ERR_INVALID_ARG;
    if (desc->batch * desc->channels > kMaxElems / desc->modes) return HM_ERR_INVALID_ARG;
    return HM_OK;
}

hm::OpShape shape_of(const hm_desc *desc) {
    hm::OpShape s;
    s.B = desc->batch;
    s.D = desc->channels;
    s.H = desc->heads;
    s.d = desc->modes;
    s.P = desc->channels / desc->heads;
    s.act = desc->act_dtype == HM_BF16 ? hm::kBF16 : hm::kF32;
    s.poles = reinterpret_cast<const float2 *>(desc->poles);
    s.residues = reinterpret_cast<const float2 *>(desc->residues);
    s.skip = desc->skip;
    return s;
}

int elem_bytes(const hm_desc *desc) { return desc->act_dtype == HM_BF16 ? 2 : 4; }

hm_status check_act(const hm_desc *desc, const void *p) {
    if (!p) return HM_ERR_INVALID_ARG;
    if (!aligned(p, (uintptr_t)elem_bytes(desc))) return HM_ERR_UNSUPPORTED;
    return HM_OK;
}

hm_status check_chunk(int64_t chunk) {
    if (chunk < 0) return HM_ERR_INVALID_ARG;
    if (chunk > 0 && chunk % 64 != 0) return HM_ERR_UNSUPPORTED;
    return HM_OK;
}

hm_status check_opts(const hm_prefill_opts *opts, int64_t *chunk, int *algo) {
    *chunk = 0;
    *algo = hm::kAlgoAuto;
    if (!opts) return HM_OK;
    hm_status st = check_chunk(opts->chunk);
    if (st != HM_OK) return st;
    if (opts->algo != HM_PREFILL_AUTO && opts->algo != HM_PREFILL_SCAN && opts->algo != HM_PREFILL_MFMA)
        return HM_ERR_INVALID_ARG;
    *chunk = opts->chunk;
    *algo = opts->algo == HM_PREFILL_SCAN ? hm::kAlgoScan : opts->algo == HM_PREFILL_MFMA ? hm::kAlgoMfma
                                                                                              : hm::kAlgoAuto;
    return HM_OK;
}

// use_scratch: take the workspace from the per-device `scratch` array instead
// of the caller (workspace and ws_bytes are then ignored).
hm_status prefill_impl(const hm_desc *desc, int64_t L, const void *q, const void *k, const void *v,
                       int64_t ld_in, void *y, int64_t ld_y, const float *state_in, float *state_out,
                       void *workspace, size_t ws_bytes, void *stream, const hm_prefill_opts *opts,
                       bool use_scratch = false) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    int64_t chunk;
    int algo;
    if ((st = check_opts(opts, &chunk, &algo)) != HM_OK) return st;
    if (L < 0 || L > kMaxElems) return HM_ERR_INVALID_ARG;
    const hm::OpShape s = shape_of(desc);
    if (s.B > 0 && L > 0) {
        if ((st = check_act(desc, q)) != HM_OK || (st = check_act(desc, k)) != HM_OK ||
            (st = check_act(desc, v)) != HM_OK || (st = check_act(desc, y)) != HM_OK)
            return st;
        if (ld_in < s.D || ld_y < s.D) return HM_ERR_INVALID_ARG;
        if (s.B * L > kMaxElems / ld_in || s.B * L > kMaxElems / ld_y) return HM_ERR_INVALID_ARG;
    }
    if (s.B > 0) {
        if (!state_out) return HM_ERR_INVALID_ARG;
        if (!aligned(state_out, 8) || (state_in && !aligned(state_in, 8))) return HM_ERR_UNSUPPORTED;
    }
    const hm::PrefillPlan plan = hm::make_prefill_plan(s, L, chunk, algo);
    // grid limits: batch rows and chunks map to the y/z launch dimensions
    if (s.B > 65535 || plan.NC > 65535) return HM_ERR_UNSUPPORTED;
    if (algo == hm::kAlgoMfma && s.B > 0 && L > 0) {
        // the matrix-core path was asked for explicitly: shape and alignment must allow it
        const int esz = elem_bytes(desc);
        if (plan.algo != hm::kAlgoMfma || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
            !aligned(y, 16) || (ld_in * esz) % 16 != 0 || (ld_y * esz) % 16 != 0)
            return HM_ERR_UNSUPPORTED;
    }
    if (use_scratch) {
        if (s.B > 0 && plan.bytes > (size_t)HM_NOALLOC_SCRATCH_BYTES) return HM_ERR_WORKSPACE;
    } else if (s.B > 0 && plan.bytes > 0) {
        if (!workspace || ws_bytes < plan.bytes) return HM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return HM_ERR_UNSUPPORTED;
    }
    if (s.B == 0) return HM_OK;
    if (use_scratch && (st = scratch_for_current_device(&workspace)) != HM_OK) return st;
    hm::PrefillArgs a;
    a.s = s;
    a.plan = plan;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_in = ld_in;
    a.y = y;
    a.ld_y = ld_y;
    a.state_in = reinterpret_cast<const float2 *>(state_in);
    a.state_out = reinterpret_cast<float2 *>(state_out);
    a.ws = static_cast<unsigned char *>(workspace);
    const hipError_t err = hm::launch_prefill(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status workspace_impl(const hm_desc *desc, int64_t L, const hm_prefill_opts *opts, size_t *bytes) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    int64_t chunk;
    int algo;
    if ((st = check_opts(opts, &chunk, &algo)) != HM_OK) return st;
    if (!bytes || L < 0 || L > kMaxElems) return HM_ERR_INVALID_ARG;
    *bytes = desc->batch > 0 ? hm::make_prefill_plan(shape_of(desc), L, chunk, algo).bytes : 0;
    return HM_OK;
}

hm_status plan_impl(const hm_desc *desc, int64_t L, const hm_prefill_opts *opts, hm_prefill_info *info) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    int64_t chunk;
    int algo;
    if ((st = check_opts(opts, &chunk, &algo)) != HM_OK) return st;
    if (!info || L < 0 || L > kMaxElems) return HM_ERR_INVALID_ARG;
    const hm::PrefillPlan plan = hm::make_prefill_plan(shape_of(desc), L, chunk, algo);
    if (algo == hm::kAlgoMfma && plan.algo != hm::kAlgoMfma) return HM_ERR_UNSUPPORTED;
    info->algo = plan.algo == hm::kAlgoMfma ? HM_PREFILL_MFMA : HM_PREFILL_SCAN;
    info->channel_tile = plan.algo == hm::kAlgoMfma ? hm::mfma_channel_tile(shape_of(desc)) : 0;
    info->chunk = plan.T;
    info->n_chunks = plan.NC;
    info->workspace_bytes = desc->batch > 0 ? plan.bytes : 0;
    return HM_OK;
}

}  // namespace

extern "C" {

int hm_abi_version(void) { return HM_ABI_VERSION; }

const char *hm_status_string(hm_status status) {
    switch (status) {
        case HM_OK: return "HM_OK";
        case HM_ERR_INVALID_ARG: return "HM_ERR_INVALID_ARG: invalid argument";
        case HM_ERR_UNSUPPORTED: return "HM_ERR_UNSUPPORTED: unsupported dtype, size or alignment";
        case HM_ERR_WORKSPACE: return "HM_ERR_WORKSPACE: workspace missing or too small";
        case HM_ERR_HIP: return "HM_ERR_HIP: kernel launch failed";
    }
    return "unknown hm_status";
}

hm_status hyena_modal_prefill_workspace(const hm_desc *desc, int64_t L, size_t *bytes) {
    return workspace_impl(desc, L, nullptr, bytes);
}

hm_status hyena_modal_prefill_workspace_ex(const hm_desc *desc, int64_t L, const hm_prefill_opts *opts,
                                           size_t *bytes) {
    return workspace_impl(desc, L, opts, bytes);
}

hm_status hyena_modal_prefill_plan(const hm_desc *desc, int64_t L, const hm_prefill_opts *opts,
                                   hm_prefill_info *info) {
    return plan_impl(desc, L, opts, info);
}

hm_status hyena_modal_prefill(const hm_desc *desc, int64_t L, const void *q, const void *k,
                              const void *v, int64_t ld_in, void *y, int64_t ld_y,
                              const float *state_in, float *state_out, void *workspace,
                              size_t ws_bytes, void *stream) {
    return prefill_impl(desc, L, q, k, v, ld_in, y, ld_y, state_in, state_out, workspace, ws_bytes,
                        stream, nullptr);
}

hm_status hyena_modal_prefill_ex(const hm_desc *desc, int64_t L, const void *q, const void *k,
                                 const void *v, int64_t ld_in, void *y, int64_t ld_y,
                                 const float *state_in, float *state_out, void *workspace,
                                 size_t ws_bytes, const hm_prefill_opts *opts, void *stream) {
    return prefill_impl(desc, L, q, k, v, ld_in, y, ld_y, state_in, state_out, workspace, ws_bytes,
                        stream, opts);
}

hm_status hyena_modal_prefill_noalloc(const hm_desc *desc, int64_t L, const void *q, const void *k,
                                      const void *v, int64_t ld_in, void *y, int64_t ld_y,
                                      const float *state_in, float *state_out,
                                      const hm_prefill_opts *opts, void *stream) {
    return prefill_impl(desc, L, q, k, v, ld_in, y, ld_y, state_in, state_out, nullptr, 0, stream, opts,
                        /*use_scratch=*/true);
}

hm_status hyena_modal_decode_step(const hm_desc *desc, const void *q, const void *k, const void *v,
                                  int64_t ld_in, void *y, int64_t ld_y, float *state, void *stream) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    const hm::OpShape s = shape_of(desc);
    if (s.B == 0) return HM_OK;
    if ((st = check_act(desc, q)) != HM_OK || (st = check_act(desc, k)) != HM_OK ||
        (st = check_act(desc, v)) != HM_OK || (st = check_act(desc, y)) != HM_OK)
        return st;
    if (!state) return HM_ERR_INVALID_ARG;
    if (!aligned(state, 8)) return HM_ERR_UNSUPPORTED;
    if (ld_in < s.D || ld_y < s.D) return HM_ERR_INVALID_ARG;
    if (s.B > kMaxElems / ld_in || s.B > kMaxElems / ld_y) return HM_ERR_INVALID_ARG;
    if (s.B > 65535 || s.D * 4 > INT32_MAX) return HM_ERR_UNSUPPORTED;  // grid limits
    hm::DecodeArgs a;
    a.s = s;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_in = ld_in;
    a.y = y;
    a.ld_y = ld_y;
    a.state = reinterpret_cast<float2 *>(state);
    const hipError_t err = hm::launch_decode_step(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_filter_materialize(const hm_desc *desc, int64_t L, float *h_out, void *stream) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (L < 0 || L > kMaxElems / desc->heads) return HM_ERR_INVALID_ARG;
    if (L == 0) return HM_OK;
    // grid limit: one workgroup per head and (at least) 128 taps
    if ((L + 127) / 128 > (int64_t)INT32_MAX / desc->heads) return HM_ERR_UNSUPPORTED;
    if (!h_out) return HM_ERR_INVALID_ARG;
    if (!aligned(h_out, 4)) return HM_ERR_UNSUPPORTED;
    hm::FilterArgs a;
    a.s = shape_of(desc);
    a.L = L;
    a.h = h_out;
    const hipError_t err = hm::launch_filter(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

static hm_status fir_check(const hm_desc *desc, const void *cache, int64_t cache_len) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (cache_len < 1 || desc->batch > kMaxElems / cache_len || desc->batch * cache_len > kMaxElems / desc->channels)
        return HM_ERR_INVALID_ARG;
    if (desc->batch > 0 && !cache) return HM_ERR_INVALID_ARG;
    if (desc->channels % 8 != 0 || (desc->channels / desc->heads) % 8 != 0) return HM_ERR_UNSUPPORTED;
    if (desc->batch > 0 && !aligned(cache, 16)) return HM_ERR_UNSUPPORTED;
    return HM_OK;
}

hm_status hyena_fir_workspace(const hm_desc *desc, size_t *bytes) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (!bytes) return HM_ERR_INVALID_ARG;
    *bytes = (size_t)hm::fir_ranges(desc->batch, desc->channels) * desc->batch * desc->channels * sizeof(float);
    return HM_OK;
}

hm_status hyena_fir_cache_fill(const hm_desc *desc, int64_t L, const void *k, const void *v, int64_t ld_in,
                               void *u_cache, int64_t cache_len, void *stream) {
    hm_status st = fir_check(desc, u_cache, cache_len);
    if (st != HM_OK) return st;
    if (L < 0 || L > cache_len) return HM_ERR_INVALID_ARG;
    if (desc->batch == 0 || L == 0) return HM_OK;
    if ((st = check_act(desc, k)) != HM_OK || (st = check_act(desc, v)) != HM_OK) return st;
    if (ld_in < desc->channels || desc->batch * L > kMaxElems / ld_in) return HM_ERR_INVALID_ARG;
    hm::FirArgs a{};
    a.s = shape_of(desc);
    a.k = k;
    a.v = v;
    a.ld_in = ld_in;
    a.cache = u_cache;
    a.cache_len = cache_len;
    const hipError_t err = hm::launch_fir_fill(a, L, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

static hm_status fir_decode_impl(const hm_desc *desc, const float *h, int64_t h_len, int64_t window, int64_t t,
                                 const void *q, const void *k, const void *v, int64_t ld_in, void *y,
                                 int64_t ld_y, void *u_cache, int64_t cache_len, void *workspace,
                                 size_t ws_bytes, int32_t loads, void *stream) {
    hm_status st = fir_check(desc, u_cache, cache_len);
    if (st != HM_OK) return st;
    if (loads < 0 || loads > 2) return HM_ERR_INVALID_ARG;
    // float32 non-temporal loads need the 512-channel block split
    if (loads == 2 && desc->act_dtype == HM_F32 && desc->channels % 512 != 0) return HM_ERR_UNSUPPORTED;
    if (t < 0 || t >= cache_len || window < 0) return HM_ERR_INVALID_ARG;
    const int64_t taps = (window == 0 || window > t + 1) ? t + 1 : window;
    if (!h || h_len < taps || h_len > kMaxElems / desc->heads) return HM_ERR_INVALID_ARG;
    if (!aligned(h, 4)) return HM_ERR_UNSUPPORTED;
    if (desc->batch == 0) return HM_OK;
    if ((st = check_act(desc, q)) != HM_OK || (st = check_act(desc, k)) != HM_OK ||
        (st = check_act(desc, v)) != HM_OK || (st = check_act(desc, y)) != HM_OK)
        return st;
    if (ld_in < desc->channels || ld_y < desc->channels) return HM_ERR_INVALID_ARG;
    if (desc->batch > kMaxElems / ld_in || desc->batch > kMaxElems / ld_y) return HM_ERR_INVALID_ARG;
    if (desc->batch > 65535) return HM_ERR_UNSUPPORTED;  // grid z
    const int R = hm::fir_ranges(desc->batch, desc->channels);
    const size_t need = (size_t)R * desc->batch * desc->channels * sizeof(float);
    if (!workspace || ws_bytes < need) return HM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HM_ERR_UNSUPPORTED;
    hm::FirArgs a{};
    a.s = shape_of(desc);
    a.h = h;
    a.h_len = h_len;
    a.t = t;
    a.lo = t + 1 - taps;
    a.R = R;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_in = ld_in;
    a.y = y;
    a.ld_y = ld_y;
    a.cache = u_cache;
    a.cache_len = cache_len;
    a.part = static_cast<float *>(workspace);
    a.loads = loads;
    const hipError_t err = hm::launch_fir_decode(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_fir_decode_step(const hm_desc *desc, const float *h, int64_t h_len, int64_t window, int64_t t,
                                const void *q, const void *k, const void *v, int64_t ld_in, void *y,
                                int64_t ld_y, void *u_cache, int64_t cache_len, void *workspace,
                                size_t ws_bytes, void *stream) {
    return fir_decode_impl(desc, h, h_len, window, t, q, k, v, ld_in, y, ld_y, u_cache, cache_len, workspace,
                           ws_bytes, HM_FIR_LOADS_AUTO, stream);
}

hm_status hyena_fir_decode_step_ex(const hm_desc *desc, const float *h, int64_t h_len, int64_t window, int64_t t,
                                   const void *q, const void *k, const void *v, int64_t ld_in, void *y,
                                   int64_t ld_y, void *u_cache, int64_t cache_len, void *workspace,
                                   size_t ws_bytes, int32_t loads, void *stream) {
    return fir_decode_impl(desc, h, h_len, window, t, q, k, v, ld_in, y, ld_y, u_cache, cache_len, workspace,
                           ws_bytes, loads, stream);
}

static size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

// FFT-prefill workspace: taps [H][L] fp32 | twiddles [N/2] | spectra [H][N] (complex fp32)
// | past N = 8192, the multi-pass work buffer [B][N][D/2] (complex fp32).
static size_t fft_workspace_bytes(const hm_desc *desc, int64_t L, size_t *off_tw, size_t *off_spec,
                                  size_t *off_z) {
    const int logn = hm::fft_log_n(L);
    const size_t N = size_t(1) << logn;
    *off_tw = align_up((size_t)desc->heads * L * sizeof(float));
    *off_spec = align_up(*off_tw + N / 2 * 8);
    *off_z = align_up(*off_spec + (size_t)desc->heads * N * 8);
    if (logn <= hm::kFftMaxLogN) return *off_z;
    return *off_z + (size_t)desc->batch * N * (size_t)(desc->channels / 2) * 8;
}

static constexpr int64_t kFftMaxL = int64_t(1) << (hm::kFftMaxLogNLong - 1);

// the multi-pass work buffer (B x N x D/2 complex) must stay addressable
static bool fft_long_fits(const hm_desc *desc, int64_t L) {
    const int logn = hm::fft_log_n(L);
    if (logn <= hm::kFftMaxLogN) return true;
    return desc->batch * (desc->channels / 2) <= kMaxElems / (int64_t(1) << logn);
}

hm_status hyena_fft_prefill_workspace(const hm_desc *desc, int64_t L, size_t *bytes) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (!bytes || L < 0) return HM_ERR_INVALID_ARG;
    if (L > kFftMaxL || (L > 0 && !fft_long_fits(desc, L))) return HM_ERR_UNSUPPORTED;
    size_t a, b, c;
    *bytes = L == 0 ? 0 : fft_workspace_bytes(desc, L, &a, &b, &c);
    return HM_OK;
}

hm_status hyena_fft_prefill(const hm_desc *desc, int64_t L, const void *q, const void *k, const void *v,
                            int64_t ld_in, void *y, int64_t ld_y, void *workspace, size_t ws_bytes, void *stream) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (L < 0) return HM_ERR_INVALID_ARG;
    if (L > kFftMaxL) return HM_ERR_UNSUPPORTED;
    if (desc->batch == 0 || L == 0) return HM_OK;
    if (!fft_long_fits(desc, L)) return HM_ERR_UNSUPPORTED;
    if ((desc->channels / desc->heads) % 2 != 0) return HM_ERR_UNSUPPORTED;  // channel pairs within a head
    if (desc->batch > 65535 || desc->channels / 2 > INT32_MAX) return HM_ERR_UNSUPPORTED;
    if ((st = check_act(desc, q)) != HM_OK || (st = check_act(desc, k)) != HM_OK ||
        (st = check_act(desc, v)) != HM_OK || (st = check_act(desc, y)) != HM_OK)
        return st;
    if (ld_in < desc->channels || ld_y < desc->channels) return HM_ERR_INVALID_ARG;
    if (desc->batch * L > kMaxElems / ld_in || desc->batch * L > kMaxElems / ld_y) return HM_ERR_INVALID_ARG;
    size_t off_tw, off_spec, off_z;
    const size_t need = fft_workspace_bytes(desc, L, &off_tw, &off_spec, &off_z);
    if (!workspace || ws_bytes < need) return HM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HM_ERR_UNSUPPORTED;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    hm::FftArgs a{};
    a.s = shape_of(desc);
    a.L = L;
    a.logn = hm::fft_log_n(L);
    a.np = hm::fft_pairs_per_group(a.s.P, a.logn);
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_in = ld_in;
    a.y = y;
    a.ld_y = ld_y;
    a.h = reinterpret_cast<float *>(ws);
    a.tw = reinterpret_cast<float2 *>(ws + off_tw);
    a.spec = reinterpret_cast<float2 *>(ws + off_spec);
    a.z = a.logn > hm::kFftMaxLogN ? reinterpret_cast<float2 *>(ws + off_z) : nullptr;
    hm::FilterArgs f;
    f.s = a.s;
    f.L = L;
    f.h = a.h;
    hipError_t err = hm::launch_filter(f, static_cast<hipStream_t>(stream));
    if (err == hipSuccess) err = hm::launch_fft_prefill(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

// Distillation workspace: residual [H][L] f64 | loss partials [H][tiles] f64 | gradient partials [H*d][chunks][4] f64.
static size_t distill_layout(const hm_desc *desc, int64_t L, size_t *off_loss, size_t *off_grad, int *tiles,
                             int *chunks) {
    *tiles = hm::distill_tiles(L, desc->modes);
    *chunks = (int)((L + hm::kDistillTile - 1) / hm::kDistillTile);
    *off_loss = align_up((size_t)desc->heads * L * sizeof(double));
    *off_grad = align_up(*off_loss + (size_t)desc->heads * *tiles * sizeof(double));
    return *off_grad + (size_t)desc->heads * desc->modes * *chunks * 4 * sizeof(double);
}

static bool distill_l_ok(const hm_desc *desc, int64_t L) {
    return L >= 1 && L <= kMaxElems / desc->heads && (L + hm::kDistillTile - 1) / hm::kDistillTile <= 65535 &&
           (int64_t)desc->heads * ((L + 127) / 128) <= INT32_MAX;
}

hm_status hyena_distill_workspace(const hm_desc *desc, int64_t L, size_t *bytes) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (!bytes || !distill_l_ok(desc, L)) return HM_ERR_INVALID_ARG;
    size_t a, b;
    int t, c;
    *bytes = distill_layout(desc, L, &a, &b, &t, &c);
    return HM_OK;
}

hm_status hyena_distill_grad(const hm_desc *desc, int64_t L, const float *h_target, float *loss, float *g_poles,
                             float *g_res, float *g_skip, void *workspace, size_t ws_bytes, void *stream) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (!distill_l_ok(desc, L)) return HM_ERR_INVALID_ARG;
    if (!h_target || !loss || !g_poles || !g_res || !g_skip) return HM_ERR_INVALID_ARG;
    if (!aligned(h_target, 4) || !aligned(loss, 4) || !aligned(g_poles, 4) || !aligned(g_res, 4) ||
        !aligned(g_skip, 4))
        return HM_ERR_UNSUPPORTED;
    hm::DistillArgs a{};
    size_t off_loss, off_grad;
    const size_t need = distill_layout(desc, L, &off_loss, &off_grad, &a.tiles, &a.chunks);
    if (!workspace || ws_bytes < need) return HM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HM_ERR_UNSUPPORTED;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.s = shape_of(desc);
    a.L = L;
    a.target = h_target;
    a.e = reinterpret_cast<double *>(ws);
    a.loss_part = reinterpret_cast<double *>(ws + off_loss);
    a.grad_part = reinterpret_cast<double *>(ws + off_grad);
    a.loss = loss;
    a.g_poles = g_poles;
    a.g_res = g_res;
    a.g_skip = g_skip;
    const hipError_t err = hm::launch_distill_grad(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_distill_adam_step(int64_t H, int64_t d, float *poles, float *residues, float *skip,
                                  const float *g_poles, const float *g_res, const float *g_skip, float *m, float *v,
                                  int64_t step, float lr, float beta1, float beta2, float eps, float r_max,
                                  void *stream) {
    if (H < 1 || d < 1 || d > HM_MAX_MODES || H > INT32_MAX / 64) return HM_ERR_INVALID_ARG;
    if (!poles || !residues || !skip || !g_poles || !g_res || !g_skip || !m || !v) return HM_ERR_INVALID_ARG;
    if (step < 1 || !(lr > 0.f) || !(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f) ||
        !(eps > 0.f) || !(r_max > 0.f && r_max < 1.f))
        return HM_ERR_INVALID_ARG;
    for (const void *p : {(const void *)poles, (const void *)residues, (const void *)skip, (const void *)g_poles,
                          (const void *)g_res, (const void *)g_skip, (const void *)m, (const void *)v})
        if (!aligned(p, 4)) return HM_ERR_UNSUPPORTED;
    hm::AdamArgs a;
    a.H = H;
    a.d = d;
    a.poles = poles;
    a.residues = residues;
    a.skip = skip;
    a.g_poles = g_poles;
    a.g_res = g_res;
    a.g_skip = g_skip;
    a.m = m;
    a.v = v;
    a.lr = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = eps;
    a.r_max = r_max;
    a.bc1 = (float)(1.0 - std::pow((double)beta1, (double)step));
    a.bc2 = (float)(1.0 - std::pow((double)beta2, (double)step));
    const hipError_t err = hm::launch_distill_adam(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_row_rms(const void *x, int64_t M, int64_t D, int64_t ld, float eps, float *inv_rms,
                        void *stream) {
    if (M < 0 || D < 1 || ld < D || M > kMaxElems / ld || !(eps >= 0.0f)) return HM_ERR_INVALID_ARG;
    if (M == 0) return HM_OK;
    if (!x || !inv_rms) return HM_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(inv_rms, 4)) return HM_ERR_UNSUPPORTED;
    if (M > int64_t(UINT32_MAX) * 4) return HM_ERR_UNSUPPORTED;
    hm::RmsArgs a;
    a.x = x;
    a.M = M;
    a.D = D;
    a.ld = ld;
    a.eps = eps;
    a.inv_rms = inv_rms;
    a.vec = aligned(x, 16) && D % 8 == 0 && ld % 8 == 0;
    const hipError_t err = hm::launch_row_rms(a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

static hm_status dense_impl(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *W, int64_t ldw,
                     const float *row_scale, bool rms, float eps, void *C, int64_t ldc, void *workspace,
                     size_t ws_bytes, void *stream) {
    if (M < 0 || N < 0 || K < 1) return HM_ERR_INVALID_ARG;
    if (lda < K || ldw < K || ldc < N) return HM_ERR_INVALID_ARG;
    if (M > kMaxElems / lda || N > kMaxElems / ldw || M > kMaxElems / (ldc > 0 ? ldc : 1))
        return HM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return HM_OK;
    if (!A || !W || !C) return HM_ERR_INVALID_ARG;
    if (K % 64 != 0 || lda % 8 != 0 || ldw % 8 != 0) return HM_ERR_UNSUPPORTED;
    if (!aligned(A, 16) || !aligned(W, 16) || !aligned(C, 2) || (row_scale && !aligned(row_scale, 4)))
        return HM_ERR_UNSUPPORTED;
    if (((M + 127) / 128) * ((N + 255) / 256) > INT32_MAX) return HM_ERR_UNSUPPORTED;
    const size_t ws_need = hm::splitk_workspace_bytes(M, N, K);
    if (workspace && ws_need > 0) {
        if (ws_bytes < ws_need) return HM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return HM_ERR_UNSUPPORTED;
    }
    hm::GemmArgs g;
    g.M = M;
    g.N = N;
    g.K = K;
    g.A = A;
    g.lda = lda;
    g.W = W;
    g.ldw = ldw;
    g.row_scale = row_scale;
    g.C = C;
    g.ldc = ldc;
    g.rms = rms;
    g.rms_eps = eps;
    g.ws = (workspace && ws_need > 0) ? static_cast<unsigned char *>(workspace) : nullptr;
    g.ws_bytes = ws_bytes;
    const hipError_t err = hm::launch_gemm(g, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_dense_bf16(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *W,
                           int64_t ldw, const float *row_scale, void *C, int64_t ldc, void *stream) {
    return dense_impl(M, N, K, A, lda, W, ldw, row_scale, false, 0.0f, C, ldc, nullptr, 0, stream);
}

hm_status hyena_dense_rms_bf16(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *W,
                               int64_t ldw, float eps, void *C, int64_t ldc, void *stream) {
    if (!(eps >= 0.0f)) return HM_ERR_INVALID_ARG;
    return dense_impl(M, N, K, A, lda, W, ldw, nullptr, true, eps, C, ldc, nullptr, 0, stream);
}

hm_status hyena_dense_workspace(int64_t M, int64_t N, int64_t K, size_t *bytes) {
    if (!bytes || M < 0 || N < 0 || K < 1) return HM_ERR_INVALID_ARG;
    *bytes = hm::splitk_workspace_bytes(M, N, K);
    return HM_OK;
}

hm_status hyena_dense_bf16_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *W,
                              int64_t ldw, const float *row_scale, void *C, int64_t ldc, void *workspace,
                              size_t ws_bytes, void *stream) {
    return dense_impl(M, N, K, A, lda, W, ldw, row_scale, false, 0.0f, C, ldc, workspace, ws_bytes, stream);
}

hm_status hyena_dense_rms_bf16_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *W,
                                  int64_t ldw, float eps, void *C, int64_t ldc, void *workspace, size_t ws_bytes,
                                  void *stream) {
    if (!(eps >= 0.0f)) return HM_ERR_INVALID_ARG;
    return dense_impl(M, N, K, A, lda, W, ldw, nullptr, true, eps, C, ldc, workspace, ws_bytes, stream);
}

hm_status hyena_pack_in_proj_bf16(int64_t D, int64_t K, const void *w_in, int64_t ldw, void *w_packed,
                                  void *stream) {
    if (D < 0 || K < 1 || ldw < K) return HM_ERR_INVALID_ARG;
    if (D == 0) return HM_OK;
    if (!w_in || !w_packed) return HM_ERR_INVALID_ARG;
    if (D % 16 != 0 || K % 8 != 0 || ldw % 8 != 0) return HM_ERR_UNSUPPORTED;
    if (!aligned(w_in, 16) || !aligned(w_packed, 16)) return HM_ERR_UNSUPPORTED;
    if (3 * D > INT32_MAX || 3 * D > kMaxElems / ldw) return HM_ERR_INVALID_ARG;
    const hipError_t err = hm::launch_pack_in_proj(D, K, w_in, ldw, w_packed, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

// ------------------------------------------------------------------ generation step, deferred state

static hm_status prep_of(const hm_desc *desc, float *state, const float *u_prev, float *rho, hm::PrepArgs *p) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    const hm::OpShape s = shape_of(desc);
    if (s.B > 0 && (!state || !u_prev || !rho)) return HM_ERR_INVALID_ARG;
    if (!hm::prepare_supported(s.d) || s.P % 2 != 0) return HM_ERR_UNSUPPORTED;
    if (s.B > 0 && (!aligned(state, 16) || !aligned(u_prev, 8) || !aligned(rho, 8))) return HM_ERR_UNSUPPORTED;
    p->B = s.B;
    p->D = s.D;
    p->H = s.H;
    p->P = s.P;
    p->d = s.d;
    p->state = reinterpret_cast<float2 *>(state);
    p->u_prev = u_prev;
    p->rho = rho;
    p->poles = s.poles;
    p->residues = s.residues;
    return HM_OK;
}

hm_status hyena_decode_prepare(const hm_desc *desc, float *state, const float *u_prev, float *rho, void *stream) {
    hm::PrepArgs p;
    hm_status st = prep_of(desc, state, u_prev, rho, &p);
    if (st != HM_OK) return st;
    if (p.B == 0) return HM_OK;
    const hipError_t err = hm::launch_prepare(p, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_layer_gate_bf16(const hm_desc *desc, const void *x, int64_t ldx, const void *w_packed, float eps,
                                const float *rho, float *u_prev, void *y, int64_t ld_y, const hm_desc *next,
                                float *next_state, const float *next_u_prev, float *next_rho, void *stream) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (!(eps >= 0.0f)) return HM_ERR_INVALID_ARG;
    hm::GemmArgs g;
    if (next && (st = prep_of(next, next_state, next_u_prev, next_rho, &g.prep)) != HM_OK) return st;
    const hm::OpShape s = shape_of(desc);
    if (s.B == 0) {
        if (g.prep.B == 0) return HM_OK;
        const hipError_t err = hm::launch_prepare(g.prep, static_cast<hipStream_t>(stream));
        return err == hipSuccess ? HM_OK : HM_ERR_HIP;
    }
    if (!x || !w_packed || !rho || !u_prev || !y) return HM_ERR_INVALID_ARG;
    if (ldx < s.D || ld_y < s.D) return HM_ERR_INVALID_ARG;
    if (s.act != hm::kBF16 || s.B > 64 || s.D != 2048 || s.P % 16 != 0) return HM_ERR_UNSUPPORTED;
    if (ldx % 8 != 0 || ld_y % 2 != 0) return HM_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(y, 4) || !aligned(rho, 8) || !aligned(u_prev, 8))
        return HM_ERR_UNSUPPORTED;
    g.M = s.B;
    g.N = 3 * s.D;
    g.K = s.D;
    g.A = x;
    g.lda = ldx;
    g.W = w_packed;
    g.ldw = s.D;
    g.row_scale = nullptr;
    g.C = nullptr;
    g.ldc = 0;
    g.rms = true;
    g.rms_eps = eps;
    g.skip = s.skip;
    g.P = s.P;
    g.H = s.H;
    g.y = y;
    g.ld_y = ld_y;
    g.rho = rho;
    g.u_prev = u_prev;
    const hipError_t err = hm::launch_layer_gate(g, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_layer_step_bf16(const hm_desc *desc, const void *x, int64_t ldx, const void *w_packed, float eps,
                                float *state, void *y, int64_t ld_y, void *stream) {
    hm_status st = check_desc(desc);
    if (st != HM_OK) return st;
    if (!(eps >= 0.0f)) return HM_ERR_INVALID_ARG;
    const hm::OpShape s = shape_of(desc);
    if (s.B == 0) return HM_OK;
    if (!x || !w_packed || !state || !y) return HM_ERR_INVALID_ARG;
    if (ldx < s.D || ld_y < s.D) return HM_ERR_INVALID_ARG;
    if (s.act != hm::kBF16 || s.B > 64 || s.D != 2048 || (s.d != 8 && s.d != 16) || s.P % 16 != 0)
        return HM_ERR_UNSUPPORTED;
    if (ldx % 8 != 0 || ld_y % 2 != 0) return HM_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(state, 16) || !aligned(y, 4))
        return HM_ERR_UNSUPPORTED;
    hm::GemmArgs g;
    g.M = s.B;
    g.N = 3 * s.D;
    g.K = s.D;
    g.A = x;
    g.lda = ldx;
    g.W = w_packed;
    g.ldw = s.D;
    g.row_scale = nullptr;
    g.C = nullptr;
    g.ldc = 0;
    g.rms = true;
    g.rms_eps = eps;
    g.state = reinterpret_cast<float2 *>(state);
    g.poles = s.poles;
    g.residues = s.residues;
    g.skip = s.skip;
    g.P = s.P;
    g.H = s.H;
    g.y = y;
    g.ld_y = ld_y;
    const hipError_t err = hm::launch_layer_step(g, (int)s.d, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? HM_OK : HM_ERR_HIP;
}

static hm_status check_linattn(const hm_linattn_desc *d) {
    if (!d || d->abi_version != HM_ABI_VERSION || d->reserved != 0) return HM_ERR_INVALID_ARG;
    if (d->act_dtype != HM_F32 && d->act_dtype != HM_BF16) return HM_ERR_UNSUPPORTED;
    if (d->batch < 0 || d->heads < 1 || d->q_heads < 1 || d->k_heads < 1 || d->v_heads < 1 || d->key_dim < 1 ||
        d->value_dim < 1 || !std::isfinite(d->scale))
        return HM_ERR_INVALID_ARG;
    if (d->heads % d->q_heads != 0 || d->heads % d->k_heads != 0 || d->heads % d->v_heads != 0)
        return HM_ERR_INVALID_ARG;
    if (d->key_dim > HM_LINATTN_MAX_DIM || d->value_dim > HM_LINATTN_MAX_DIM) return HM_ERR_UNSUPPORTED;
    if (d->batch > kMaxElems / d->heads || d->batch * d->heads > kMaxElems / (d->key_dim * d->value_dim))
        return HM_ERR_INVALID_ARG;
    return HM_OK;
}

static hm::LinAttnShape linattn_shape(const hm_linattn_desc *d) {
    hm::LinAttnShape s;
    s.B = d->batch;
    s.H = d->heads;
    s.qh = d->q_heads;
    s.kh = d->k_heads;
    s.vh = d->v_heads;
    s.dk = (int)d->key_dim;
    s.dv = (int)d->value_dim;
    s.act = d->act_dtype == HM_BF16 ? hm::kBF16 : hm::kF32;
    s.scale = d->scale;
    return s;
}

// Activations, decay and states of a call over L tokens (1 for a generated token).
static hm_status linattn_args(const hm_linattn_desc *d, int64_t L, const void *q, int64_t ld_q, const void *k,
                              int64_t ld_k, const void *v, int64_t ld_v, const float *decay, int64_t ld_decay,
                              void *y, int64_t ld_y, const float *state_in, float *state_out, hm::LinAttnArgs *a) {
    const uintptr_t e = d->act_dtype == HM_BF16 ? 2 : 4;
    if (L > 0) {
        if (!q || !k || !v || !y) return HM_ERR_INVALID_ARG;
        if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(y, e)) return HM_ERR_UNSUPPORTED;
        if (ld_q < d->q_heads * d->key_dim || ld_k < d->k_heads * d->key_dim || ld_v < d->v_heads * d->value_dim ||
            ld_y < d->heads * d->value_dim)
            return HM_ERR_INVALID_ARG;
        const int64_t rows = kMaxElems / L >= d->batch ? d->batch * L : kMaxElems;
        for (int64_t ld : {ld_q, ld_k, ld_v, ld_y, ld_decay})
            if (ld > 0 && rows > kMaxElems / ld) return HM_ERR_INVALID_ARG;
    }
    if (decay) {
        if (ld_decay != 0 && ld_decay < d->heads) return HM_ERR_INVALID_ARG;
        if (!aligned(decay, 4)) return HM_ERR_UNSUPPORTED;
    }
    if (!state_out) return HM_ERR_INVALID_ARG;
    if (!aligned(state_out, 4) || (state_in && !aligned(state_in, 4))) return HM_ERR_UNSUPPORTED;
    *a = hm::LinAttnArgs{};
    a->s = linattn_shape(d);
    a->L = L;
    a->q = q;
    a->k = k;
    a->v = v;
    a->ld_q = ld_q;
    a->ld_k = ld_k;
    a->ld_v = ld_v;
    a->decay = decay;
    a->ld_decay = ld_decay;
    a->y = y;
    a->ld_y = ld_y;
    a->state_in = state_in;
    a->state_out = state_out;
    return HM_OK;
}

// Rows and heads of a launch: fewer than 2^32 threads, up to four value tiles of 512
// each, rounded up to eight.
constexpr int64_t kMostHeads = (int64_t(1) << 21) - 8;

hm_status hyena_linattn_prefill_workspace(const hm_linattn_desc *desc, int64_t L, size_t *bytes) {
    hm_status st = check_linattn(desc);
    if (st != HM_OK) return st;
    if (!bytes || L < 0 || L > kMaxElems) return HM_ERR_INVALID_ARG;
    *bytes = desc->batch > 0 ? hm::linattn_workspace(linattn_shape(desc), L) : 0;
    return HM_OK;
}

hm_status hyena_linattn_prefill(const hm_linattn_desc *desc, int64_t L, const int32_t *lengths, const void *q,
                                int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                                const float *log_decay, int64_t ld_decay, void *y, int64_t ld_y,
                                const float *state_in, float *state_out, void *workspace, size_t ws_bytes,
                                void *stream) {
    hm_status st = check_linattn(desc);
    if (st != HM_OK) return st;
    if (L < 0 || L > INT32_MAX / 2) return L < 0 ? HM_ERR_INVALID_ARG : HM_ERR_UNSUPPORTED;
    if (desc->batch == 0) return HM_OK;
    hm::LinAttnArgs a;
    if ((st = linattn_args(desc, L, q, ld_q, k, ld_k, v, ld_v, log_decay, ld_decay, y, ld_y, state_in, state_out,
                           &a)) != HM_OK)
        return st;
    if (lengths && !aligned(lengths, 4)) return HM_ERR_UNSUPPORTED;
    const size_t need = hm::linattn_workspace(a.s, L);
    if (need > 0) {
        if (!workspace || ws_bytes < need) return HM_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return HM_ERR_UNSUPPORTED;
    }
    if (desc->batch * desc->heads > kMostHeads) return HM_ERR_UNSUPPORTED;
    // a chunk of 64 rows is addressed by 32-bit byte offsets
    for (int64_t ld : {ld_q, ld_k, ld_v})
        if (L > 0 && ld >= int64_t(1) << 22) return HM_ERR_UNSUPPORTED;
    a.lengths = lengths;
    a.ws = static_cast<unsigned char *>(workspace);
    return hm::launch_linattn_prefill(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_linattn_decode_step(const hm_linattn_desc *desc, const void *q, int64_t ld_q, const void *k,
                                    int64_t ld_k, const void *v, int64_t ld_v, const float *log_decay,
                                    int64_t ld_decay, void *y, int64_t ld_y, const float *state_in,
                                    const int32_t *src_rows, float *state_out, void *stream) {
    hm_status st = check_linattn(desc);
    if (st != HM_OK) return st;
    if (desc->batch == 0) return HM_OK;
    if (!state_in) return HM_ERR_INVALID_ARG;
    hm::LinAttnArgs a;
    if ((st = linattn_args(desc, 1, q, ld_q, k, ld_k, v, ld_v, log_decay, ld_decay, y, ld_y, state_in, state_out,
                           &a)) != HM_OK)
        return st;
    if (src_rows) {
        if (state_in == state_out) return HM_ERR_INVALID_ARG;
        if (!aligned(src_rows, 4)) return HM_ERR_UNSUPPORTED;
    }
    if (desc->batch * desc->heads > kMostHeads) return HM_ERR_UNSUPPORTED;
    a.src_rows = src_rows;
    return hm::launch_linattn_decode(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

// A launch has fewer than 2^32 threads: at most 2^23 rows and one segment of 8192
// logits more for each 8192 (segments are shorter only where they are few).
static hm_status check_beams(int64_t groups, int64_t beams, int64_t vocab, int64_t select) {
    if (groups < 0 || beams < 1 || vocab < 1 || select < 1 || beams > HM_BEAM_MAX || select > HM_BEAM_MAX)
        return HM_ERR_INVALID_ARG;
    // Places in a row are 32-bit: its last segment goes up to 2 * 8192 past the row's end.
    if (vocab > (INT32_MAX - (1 << 14)) / beams || groups >= (int64_t(1) << 23) / beams) return HM_ERR_UNSUPPORTED;
    if (groups * beams > (int64_t(1) << 36) / vocab) return HM_ERR_UNSUPPORTED;
    if (select > beams * vocab) return HM_ERR_INVALID_ARG;
    return HM_OK;
}

hm_status hyena_beam_select_workspace(int64_t groups, int64_t beams, int64_t vocab, int64_t select, size_t *bytes) {
    const hm_status st = check_beams(groups, beams, vocab, select);
    if (st != HM_OK) return st;
    if (!bytes) return HM_ERR_INVALID_ARG;
    *bytes = groups > 0 ? hm::beam_select_workspace(groups, beams, vocab, select) : 0;
    return HM_OK;
}

hm_status hyena_beam_select(int64_t groups, int64_t beams, int64_t vocab, int64_t select, int32_t dtype,
                            const void *logits, int64_t ld, const float *scores, const uint8_t *finished,
                            int64_t end_token, float *out_scores, int32_t *out_tokens, int32_t *out_parents,
                            uint8_t *out_finished, void *workspace, size_t ws_bytes, void *stream) {
    hm_status st = check_beams(groups, beams, vocab, select);
    if (st != HM_OK) return st;
    if (dtype != HM_F32 && dtype != HM_BF16) return HM_ERR_UNSUPPORTED;
    if (ld < vocab || end_token < -1 || end_token >= vocab || (finished && end_token < 0)) return HM_ERR_INVALID_ARG;
    if (groups == 0) return HM_OK;
    if (!logits || !scores || !out_scores || !out_tokens || !out_parents) return HM_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == HM_BF16 ? 2 : 4) || !aligned(scores, 4) || !aligned(out_scores, 4) ||
        !aligned(out_tokens, 4) || !aligned(out_parents, 4))
        return HM_ERR_UNSUPPORTED;
    if (groups * beams > kMaxElems / ld) return HM_ERR_INVALID_ARG;
    // in place, a group's would land on another's
    if ((out_scores == scores || (finished && out_finished == finished)) && select != beams) return HM_ERR_INVALID_ARG;
    const size_t need = hm::beam_select_workspace(groups, beams, vocab, select);
    if (!workspace || ws_bytes < need) return HM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return HM_ERR_UNSUPPORTED;
    hm::BeamSelectArgs a;
    a.groups = groups;
    a.beams = beams;
    a.vocab = vocab;
    a.select = select;
    a.act = dtype == HM_BF16 ? hm::kBF16 : hm::kF32;
    a.logits = logits;
    a.ld = ld;
    a.scores = scores;
    a.finished = finished;
    a.end_token = end_token;
    a.out_scores = out_scores;
    a.out_tokens = out_tokens;
    a.out_parents = out_parents;
    a.out_finished = out_finished;
    a.ws = static_cast<unsigned char *>(workspace);
    return hm::launch_beam_select(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_beam_reorder(int64_t groups, int64_t beams, const int32_t *parents, int64_t n, void *const *buffers,
                             const int64_t *row_bytes, void *stream) {
    const hm_status st = check_beams(groups, beams, 1, 1);
    if (st != HM_OK) return st;
    if (n < 0 || (n > 0 && (!buffers || !row_bytes))) return HM_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i) {
        if (row_bytes[i] < 0 || (groups > 0 && row_bytes[i] > kMaxElems / (groups * beams))) return HM_ERR_INVALID_ARG;
        if (groups > 0 && row_bytes[i] > 0 && !buffers[i]) return HM_ERR_INVALID_ARG;
    }
    if (groups == 0 || n == 0) return HM_OK;
    if (!parents) return HM_ERR_INVALID_ARG;
    if (groups > 65535) return HM_ERR_UNSUPPORTED;  // grid limits
    for (int64_t i = 0; i < n; ++i)
        if (row_bytes[i] > int64_t(1) << 33) return HM_ERR_UNSUPPORTED;  // 2^23 workgroups of single bytes
    if (!aligned(parents, 4)) return HM_ERR_UNSUPPORTED;
    return hm::launch_beam_reorder(groups, beams, parents, n, buffers, row_bytes,
                                   static_cast<hipStream_t>(stream)) == hipSuccess
               ? HM_OK
               : HM_ERR_HIP;
}

static hm_status check_recurrence(const hm_recurrence_desc *d) {
    if (!d || d->abi_version != HM_ABI_VERSION) return HM_ERR_INVALID_ARG;
    if (d->act_dtype != HM_F32 && d->act_dtype != HM_BF16) return HM_ERR_UNSUPPORTED;
    if (d->batch < 0 || d->channels < 1) return HM_ERR_INVALID_ARG;
    if (d->gate != HM_GATE_LOG && d->gate != HM_GATE_SIGMOID) return HM_ERR_INVALID_ARG;
    if (d->input != HM_GATE_INPUT_FREE && d->input != HM_GATE_INPUT_CONVEX && d->input != HM_GATE_INPUT_NORM)
        return HM_ERR_INVALID_ARG;
    if (d->batch > kMaxElems / d->channels) return HM_ERR_INVALID_ARG;
    return HM_OK;
}

// Rows of activations of `rows` tokens: pointer, alignment, stride and extent.
static hm_status check_rows(const void *p, int64_t ld, int64_t width, int64_t rows, uintptr_t e) {
    if (!p || ld < width) return HM_ERR_INVALID_ARG;
    if (!aligned(p, e)) return HM_ERR_UNSUPPORTED;
    return rows > kMaxElems / ld ? HM_ERR_INVALID_ARG : HM_OK;
}

// Sizes of a call over L tokens, and its inputs' rows.
static hm_status recurrence_args(const hm_recurrence_desc *d, int64_t L, const void *q, int64_t ld_q, const void *g,
                                 int64_t ld_g, const void *v, int64_t ld_v, hm::RecurArgs *a) {
    const uintptr_t e = d->act_dtype == HM_BF16 ? 2 : 4;
    if (L > 0) {
        const int64_t rows = kMaxElems / L >= d->batch ? d->batch * L : kMaxElems;
        hm_status st;
        if ((q && (st = check_rows(q, ld_q, d->channels, rows, e)) != HM_OK) ||
            (st = check_rows(g, ld_g, d->channels, rows, e)) != HM_OK ||
            (st = check_rows(v, ld_v, d->channels, rows, e)) != HM_OK)
            return st;
        for (int64_t ld : {q ? ld_q : 0, ld_g, ld_v})
            if (L > 1 && ld >= hm::kRecurMostStride) return HM_ERR_UNSUPPORTED;
    }
    *a = hm::RecurArgs{};
    a->B = d->batch;
    a->D = d->channels;
    a->L = L;
    a->act = d->act_dtype == HM_BF16 ? hm::kBF16 : hm::kF32;
    a->gate = d->gate == HM_GATE_LOG ? hm::kGateLog : hm::kGateSigmoid;
    a->input = d->input == HM_GATE_INPUT_FREE     ? hm::kInputFree
               : d->input == HM_GATE_INPUT_CONVEX ? hm::kInputConvex
                                                  : hm::kInputNorm;
    a->q = q;
    a->g = g;
    a->v = v;
    a->ld_q = ld_q;
    a->ld_g = ld_g;
    a->ld_v = ld_v;
    return HM_OK;
}

// Workgroups of a launch: fewer than 2^32 threads of at most 512 each.
constexpr int64_t kMostGroups = int64_t(1) << 23;

static hm_status check_recurrence_length(const hm_recurrence_desc *d, int64_t L) {
    if (L < 0) return HM_ERR_INVALID_ARG;
    if (L > INT32_MAX / 2) return HM_ERR_UNSUPPORTED;
    const int64_t tiles = (d->channels + 63) / 64, chunks = L > 0 ? (L + 63) / 64 : 1;
    if (d->batch > 0 && (tiles >= kMostGroups || chunks >= kMostGroups || tiles * chunks >= kMostGroups ||
                         d->batch >= (kMostGroups + tiles * chunks - 1) / (tiles * chunks)))
        return HM_ERR_UNSUPPORTED;
    return HM_OK;
}

static hm_status check_workspace(const void *workspace, size_t ws_bytes, size_t need) {
    if (need == 0) return HM_OK;
    if (!workspace || ws_bytes < need) return HM_ERR_WORKSPACE;
    return aligned(workspace, 256) ? HM_OK : HM_ERR_UNSUPPORTED;
}

hm_status hyena_recurrence_workspace(const hm_recurrence_desc *desc, int64_t L, size_t *bytes) {
    hm_status st = check_recurrence(desc);
    if (st != HM_OK) return st;
    if (!bytes) return HM_ERR_INVALID_ARG;
    if ((st = check_recurrence_length(desc, L)) != HM_OK) return st;
    *bytes = desc->batch > 0 ? hm::recurrence_workspace(desc->batch, desc->channels, L) : 0;
    return HM_OK;
}

hm_status hyena_recurrence_prefill(const hm_recurrence_desc *desc, int64_t L, const int32_t *lengths, const void *q,
                                   int64_t ld_q, const void *g, int64_t ld_g, const void *v, int64_t ld_v, void *y,
                                   int64_t ld_y, const float *state_in, float *state_out, float *chunk_states,
                                   void *workspace, size_t ws_bytes, void *stream) {
    hm_status st = check_recurrence(desc);
    if (st != HM_OK) return st;
    if ((st = check_recurrence_length(desc, L)) != HM_OK) return st;
    if (desc->batch == 0) return HM_OK;
    hm::RecurArgs a;
    if ((st = recurrence_args(desc, L, q, ld_q, g, ld_g, v, ld_v, &a)) != HM_OK) return st;
    if (L > 0 && (st = check_rows(y, ld_y, desc->channels, desc->batch * L, desc->act_dtype == HM_BF16 ? 2 : 4)) != HM_OK)
        return st;
    if (L > 1 && ld_y >= hm::kRecurMostStride) return HM_ERR_UNSUPPORTED;
    if (!state_out) return HM_ERR_INVALID_ARG;
    if (!aligned(state_out, 4) || !aligned(state_in, 4) || !aligned(chunk_states, 4) || !aligned(lengths, 4))
        return HM_ERR_UNSUPPORTED;
    if ((st = check_workspace(workspace, ws_bytes, hm::recurrence_workspace(a.B, a.D, L))) != HM_OK) return st;
    a.lengths = lengths;
    a.y = y;
    a.ld_y = ld_y;
    a.state_in = state_in;
    a.state_out = state_out;
    a.chunk_states = chunk_states;
    a.ws = static_cast<unsigned char *>(workspace);
    return hm::launch_recurrence_prefill(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_recurrence_backward(const hm_recurrence_desc *desc, int64_t L, const int32_t *lengths, const void *q,
                                    int64_t ld_q, const void *g, int64_t ld_g, const void *v, int64_t ld_v,
                                    const void *dy, int64_t ld_dy, const float *chunk_states, const float *dstate_out,
                                    void *dq, int64_t ld_dq, void *dg, int64_t ld_dg, void *dv, int64_t ld_dv,
                                    float *dstate_in, void *workspace, size_t ws_bytes, void *stream) {
    hm_status st = check_recurrence(desc);
    if (st != HM_OK) return st;
    if ((st = check_recurrence_length(desc, L)) != HM_OK) return st;
    if (desc->batch == 0) return HM_OK;
    hm::RecurArgs a;
    if ((st = recurrence_args(desc, L, q, ld_q, g, ld_g, v, ld_v, &a)) != HM_OK) return st;
    if ((q == nullptr) != (dq == nullptr)) return HM_ERR_INVALID_ARG;
    if (L > 0) {
        const uintptr_t e = desc->act_dtype == HM_BF16 ? 2 : 4;
        const int64_t rows = desc->batch * L;
        if ((st = check_rows(dy, ld_dy, desc->channels, rows, e)) != HM_OK ||
            (dq && (st = check_rows(dq, ld_dq, desc->channels, rows, e)) != HM_OK) ||
            (st = check_rows(dg, ld_dg, desc->channels, rows, e)) != HM_OK ||
            (st = check_rows(dv, ld_dv, desc->channels, rows, e)) != HM_OK)
            return st;
        for (int64_t ld : {ld_dy, dq ? ld_dq : 0, ld_dg, ld_dv})
            if (L > 1 && ld >= hm::kRecurMostStride) return HM_ERR_UNSUPPORTED;
        if (!chunk_states) return HM_ERR_INVALID_ARG;
    }
    if (!aligned(chunk_states, 4) || !aligned(dstate_out, 4) || !aligned(dstate_in, 4) || !aligned(lengths, 4))
        return HM_ERR_UNSUPPORTED;
    if ((st = check_workspace(workspace, ws_bytes, hm::recurrence_workspace(a.B, a.D, L))) != HM_OK) return st;
    a.lengths = lengths;
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.chunk_states = const_cast<float *>(chunk_states);
    a.dstate_out = dstate_out;
    a.dq = dq;
    a.dg = dg;
    a.dv = dv;
    a.ld_dq = ld_dq;
    a.ld_dg = ld_dg;
    a.ld_dv = ld_dv;
    a.dstate_in = dstate_in;
    a.ws = static_cast<unsigned char *>(workspace);
    return hm::launch_recurrence_backward(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

hm_status hyena_recurrence_decode_step(const hm_recurrence_desc *desc, const void *q, int64_t ld_q, const void *g,
                                       int64_t ld_g, const void *v, int64_t ld_v, void *y, int64_t ld_y,
                                       const float *state_in, const int32_t *src_rows, float *state_out,
                                       void *stream) {
    hm_status st = check_recurrence(desc);
    if (st != HM_OK) return st;
    if (desc->batch == 0) return HM_OK;
    hm::RecurArgs a;
    if ((st = recurrence_args(desc, 1, q, ld_q, g, ld_g, v, ld_v, &a)) != HM_OK) return st;
    if ((st = check_rows(y, ld_y, desc->channels, desc->batch, desc->act_dtype == HM_BF16 ? 2 : 4)) != HM_OK) return st;
    if (!state_in || !state_out) return HM_ERR_INVALID_ARG;
    if (!aligned(state_in, 4) || !aligned(state_out, 4) || !aligned(src_rows, 4)) return HM_ERR_UNSUPPORTED;
    if (src_rows && state_in == state_out) return HM_ERR_INVALID_ARG;
    const int64_t tiles = (desc->channels + 255) / 256;
    if (desc->batch >= (kMostGroups + tiles - 1) / tiles) return HM_ERR_UNSUPPORTED;
    a.y = y;
    a.ld_y = ld_y;
    a.state_in = state_in;
    a.src_rows = src_rows;
    a.state_out = state_out;
    return hm::launch_recurrence_decode(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

// Rows and columns that 8-bit integers are held for.
static hm_status check_int8(int64_t M, int64_t K) {
    if (M < 0 || K < 1) return HM_ERR_INVALID_ARG;
    return K > HM_INT8_MAX_K || M >= INT32_MAX - 511 ? HM_ERR_UNSUPPORTED : HM_OK;
}

hm_status hyena_int8_bytes(int64_t M, int64_t K, size_t *bytes) {
    const hm_status st = check_int8(M, K);
    if (st != HM_OK) return st;
    if (!bytes) return HM_ERR_INVALID_ARG;
    *bytes = (size_t)((M + 15) / 16) * (size_t)((K + 63) / 64) * 1024;
    return HM_OK;
}

// Rows to bring to 8 bits (M > 0), but for where they go.
static hm_status check_quantize(int64_t M, int64_t K, int32_t dtype, const void *x, int64_t ldx, int32_t rms, float eps) {
    if (dtype != HM_F32 && dtype != HM_BF16) return HM_ERR_UNSUPPORTED;
    if (M >= int64_t(1) << 24) return HM_ERR_UNSUPPORTED;  // a workgroup of 256 threads a row: fewer than 2^32
    if (rms && !(std::isfinite(eps) && eps >= 0.0f)) return HM_ERR_INVALID_ARG;
    if (ldx < K) return HM_ERR_INVALID_ARG;
    return M > 0 ? check_rows(x, ldx, K, M, dtype == HM_BF16 ? 2 : 4) : HM_OK;
}

hm_status hyena_quantize_rows(int64_t M, int64_t K, int32_t dtype, const void *x, int64_t ldx, int32_t rms, float eps,
                              int8_t *q, float *scale, void *stream) {
    hm_status st = check_int8(M, K);
    if (st == HM_OK) st = check_quantize(M, K, dtype, x, ldx, rms, eps);
    if (st != HM_OK) return st;
    if (M == 0) return HM_OK;
    if (!q || !scale) return HM_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(scale, 4)) return HM_ERR_UNSUPPORTED;
    const hm::QuantArgs a{M, K, dtype == HM_BF16 ? hm::kBF16 : hm::kF32, x, ldx, rms != 0, eps, q, scale};
    return hm::launch_quantize_rows(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

// A product's sizes, weights and outputs.
static hm_status check_product(int64_t M, int64_t N, int64_t K, const int8_t *W, const float *w_scale, int32_t dtype,
                               const void *C, int64_t ldc) {
    hm_status st = check_int8(M, K);
    if (st == HM_OK) st = check_int8(N, K);
    if (st != HM_OK) return st;
    if (dtype != HM_F32 && dtype != HM_BF16) return HM_ERR_UNSUPPORTED;
    if (ldc < N) return HM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return HM_OK;
    // fewer than 2^32 threads: 512 for 256 x 256 outputs, or 256 for 16 columns of a few rows
    if ((M + 255) / 256 >= ((int64_t(1) << 20) + (N + 255) / 256 - 1) / ((N + 255) / 256)) return HM_ERR_UNSUPPORTED;
    if (!W || !w_scale || !C) return HM_ERR_INVALID_ARG;
    if (!aligned(W, 16) || !aligned(w_scale, 4) || !aligned(C, dtype == HM_BF16 ? 2 : 4)) return HM_ERR_UNSUPPORTED;
    return M > kMaxElems / ldc ? HM_ERR_INVALID_ARG : HM_OK;
}

hm_status hyena_dense_int8(int64_t M, int64_t N, int64_t K, const int8_t *A, const float *a_scale, const int8_t *W,
                           const float *w_scale, int32_t dtype, void *C, int64_t ldc, void *stream) {
    const hm_status st = check_product(M, N, K, W, w_scale, dtype, C, ldc);
    if (st != HM_OK) return st;
    if (M == 0 || N == 0) return HM_OK;
    if (!A || !a_scale) return HM_ERR_INVALID_ARG;
    if (!aligned(A, 16) || !aligned(a_scale, 4)) return HM_ERR_UNSUPPORTED;
    const hm::Int8GemmArgs a{M, N, K, A, a_scale, W, w_scale, dtype == HM_BF16 ? hm::kBF16 : hm::kF32, C, ldc};
    return hm::launch_dense_int8(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

// The rows, then their scales.
static size_t int8_rows_bytes(int64_t M, int64_t K) {
    return (size_t)((M + 15) / 16) * (size_t)((K + 63) / 64) * 1024 + ((size_t)M * sizeof(float) + 255) / 256 * 256;
}

hm_status hyena_dense_int8_rows_workspace(int64_t M, int64_t K, size_t *bytes) {
    const hm_status st = check_int8(M, K);
    if (st != HM_OK) return st;
    if (!bytes) return HM_ERR_INVALID_ARG;
    *bytes = int8_rows_bytes(M, K);
    return HM_OK;
}

// Whether M rows of `width` bytes, `pitch` apart, and M others share no byte.
static bool rows_apart(const void *a, int64_t pitch_a, int64_t width_a, const void *b, int64_t pitch_b, int64_t width_b,
                       int64_t M) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    if (p + (uintptr_t)((M - 1) * pitch_a + width_a) <= q || q + (uintptr_t)((M - 1) * pitch_b + width_b) <= p) return true;
    if (pitch_a != pitch_b) return false;
    const int64_t off = (int64_t)(q - p) % pitch_a, at = off < 0 ? off + pitch_a : off;  // columns of wider rows
    return at >= width_a && at + width_b <= pitch_a;
}

hm_status hyena_dense_int8_rows(int64_t M, int64_t N, int64_t K, int32_t x_dtype, const void *x, int64_t ldx, int32_t rms,
                                float eps, const int8_t *W, const float *w_scale, int32_t dtype, void *C, int64_t ldc,
                                void *workspace, size_t ws_bytes, void *stream) {
    hm_status st = check_product(M, N, K, W, w_scale, dtype, C, ldc);
    if (st == HM_OK) st = check_quantize(M, K, x_dtype, x, ldx, rms, eps);
    if (st != HM_OK) return st;
    if (M == 0 || N == 0) return HM_OK;
    if ((st = check_workspace(workspace, ws_bytes, int8_rows_bytes(M, K))) != HM_OK) return st;
    int8_t *q = static_cast<int8_t *>(workspace);
    float *scale = reinterpret_cast<float *>(q + (M + 15) / 16 * ((K + 63) / 64) * 1024);
    const hm::QuantArgs a{M, K, x_dtype == HM_BF16 ? hm::kBF16 : hm::kF32, x, ldx, rms != 0, eps, q, scale};
    const hm::Int8GemmArgs g{M, N, K, q, scale, W, w_scale, dtype == HM_BF16 ? hm::kBF16 : hm::kF32, C, ldc};
    const int64_t ex = x_dtype == HM_BF16 ? 2 : 4, ec = dtype == HM_BF16 ? 2 : 4;
    const bool apart = rows_apart(x, ldx * ex, K * ex, C, ldc * ec, N * ec, M);
    return hm::launch_dense_int8_rows(a, g, apart, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

static hm_status check_drafts(int64_t batch, int64_t drafts, int64_t vocab) {
    if (batch < 0 || drafts < 0 || drafts > HM_DRAFT_MAX || vocab < 1) return HM_ERR_INVALID_ARG;
    if (vocab > INT32_MAX - (1 << 14)) return HM_ERR_UNSUPPORTED;
    const int64_t parts = (vocab + 1023) / 1024;
    return batch >= (kMostGroups + parts - 1) / parts ? HM_ERR_UNSUPPORTED : HM_OK;
}

hm_status hyena_draft_verify_workspace(int64_t batch, int64_t drafts, int64_t vocab, size_t *bytes) {
    const hm_status st = check_drafts(batch, drafts, vocab);
    if (st != HM_OK) return st;
    if (!bytes) return HM_ERR_INVALID_ARG;
    *bytes = batch > 0 ? hm::draft_verify_workspace(batch, vocab) : 0;
    return HM_OK;
}

hm_status hyena_draft_verify(int64_t batch, int64_t drafts, int64_t vocab, int32_t dtype, const void *p, int64_t ld_p,
                             const void *q, int64_t ld_q, const int32_t *tokens, const int32_t *lengths, const float *u,
                             int32_t *out_tokens, int32_t *out_accepted, void *workspace, size_t ws_bytes,
                             void *stream) {
    hm_status st = check_drafts(batch, drafts, vocab);
    if (st != HM_OK) return st;
    if (dtype != HM_F32 && dtype != HM_BF16) return HM_ERR_UNSUPPORTED;
    const uintptr_t e = dtype == HM_BF16 ? 2 : 4;
    if (batch == 0) return HM_OK;
    if ((st = check_rows(p, ld_p, vocab, batch * (drafts + 1), e)) != HM_OK) return st;
    if (q && drafts > 0 && (st = check_rows(q, ld_q, vocab, batch * drafts, e)) != HM_OK) return st;
    if ((drafts > 0 && !tokens) || !u || !out_tokens || !out_accepted) return HM_ERR_INVALID_ARG;
    if (!aligned(tokens, 4) || !aligned(lengths, 4) || !aligned(u, 4) || !aligned(out_tokens, 4) ||
        !aligned(out_accepted, 4))
        return HM_ERR_UNSUPPORTED;
    if ((st = check_workspace(workspace, ws_bytes, hm::draft_verify_workspace(batch, vocab))) != HM_OK) return st;
    const hm::VerifyArgs a{batch,  (int)drafts, vocab, dtype == HM_BF16 ? hm::kBF16 : hm::kF32,
                           p,      ld_p,        q,     ld_q,
                           tokens, lengths,     u,     out_tokens,
                           out_accepted, static_cast<unsigned char *>(workspace)};
    return hm::launch_draft_verify(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HM_OK : HM_ERR_HIP;
}

}  // extern "C"
