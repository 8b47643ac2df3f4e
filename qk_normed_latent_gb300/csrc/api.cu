// C-ABI entry points: argument validation, planning and dispatch.
//
// Every call validates on the host before launching anything and returns a
// QKMLA_* code; nothing here allocates device memory except the per-device
// status word, a static __device__ variable.
#include <algorithm>
#include <mutex>

#include "common.cuh"

namespace qkmla {

__device__ int g_status_word;

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sm_count[kMaxDevices];
int* g_status_ptr[kMaxDevices];

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
}  // namespace

int device_sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_sm_count[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        g_sm_count[dev] = n;
    }
    return g_sm_count[dev];
}

int* device_status_ptr() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_status_ptr[dev] == nullptr) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
        g_status_ptr[dev] = (int*)p;
    }
    return g_status_ptr[dev];
}

static int validate_decode(const qkmla_decode_args* a, const DecodeExt& x) {
    if (!a) return QKMLA_ERR_INVALID;
    if (x.window < 0 || x.sinks < 0 || (x.sinks > 0 && x.window == 0)) return QKMLA_ERR_INVALID;
    const bool q8 = a->cache_dtype == QKMLA_E4M3;
    if (!q8 && x.kv_scale) return QKMLA_ERR_INVALID;
    const bool plain = (a->flags & QKMLA_FLAG_PLAIN_MLA) != 0;
    if (a->B < 1 || a->s_q < 1 || a->H < 1 || a->G < 1 || a->d_c < 1 || a->d_r < 0) return QKMLA_ERR_INVALID;
    if (a->H % a->G) return QKMLA_ERR_INVALID;
    if (a->page_size < 1 || a->max_pages < 1 || a->num_slots < 1 || a->num_slots % a->page_size)
        return QKMLA_ERR_INVALID;
    if ((int64_t)a->max_pages * a->page_size > INT32_MAX - 4096) return QKMLA_ERR_INVALID;   // tokens are counted as int
    if (a->num_splits < 0 || a->num_splits > 1024) return QKMLA_ERR_INVALID;
    if ((int64_t)a->B * a->s_q > INT32_MAX / a->H) return QKMLA_ERR_INVALID;   // rows are counted, and launched, as int
    if (a->cache_dtype != QKMLA_F32 && a->cache_dtype != QKMLA_BF16 && !(q8 && x.kv_scale)) return QKMLA_ERR_UNSUPPORTED;
    if (q8 && (a->d_c % 2 || !aligned(x.kv_scale, 4))) return QKMLA_ERR_INVALID;
    if (a->o_dtype != QKMLA_F32 && a->o_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    if (!a->q_tilde || !a->kv_cache || !a->seq_lens || !a->o) return QKMLA_ERR_INVALID;
    if (!plain && (!a->alpha_q || !a->ak_cache)) return QKMLA_ERR_INVALID;
    if (a->d_r > 0 && !a->q_rope) return QKMLA_ERR_INVALID;
    if (!(a->softmax_scale > 0.f) || !(a->eps >= 0.f)) return QKMLA_ERR_INVALID;
    const size_t esz = a->cache_dtype == QKMLA_F32 ? 4 : 2;
    if (!aligned(a->q_tilde, esz) || !aligned(a->kv_cache, esz) || !aligned(a->o, 4)) return QKMLA_ERR_INVALID;
    const int hpg = a->H / a->G;
    if (hpg != 1 && hpg != 2 && hpg != 4 && hpg != 8 && hpg != 16) return QKMLA_ERR_UNSUPPORTED;
    if (a->d_c > 512 || a->d_r > 128) return QKMLA_ERR_UNSUPPORTED;
    return QKMLA_OK;
}

// Split counts the tensor-core kernels are launched with: an item a CTA in the grid's y, at most 65535.
static bool tc_splits(const qkmla_decode_args* a) {
    return a->num_splits <= 256 && (int64_t)a->B * a->num_splits <= 65535;
}

int plan_decode(const qkmla_decode_args* a, const DecodeExt& x, DecodePlan* plan) {
    const int v = validate_decode(a, x);
    if (v != QKMLA_OK) return v;
    const int sms = device_sm_count();
    if (sms <= 0) return QKMLA_ERR_CUDA;
    const bool stall = (a->flags & QKMLA_FLAG_TEST_STALL) != 0;
    if (stall && x.active()) return QKMLA_ERR_UNSUPPORTED;
    if (!(a->flags & QKMLA_FLAG_FORCE_SIMT) && tc_supported(a) && tc_splits(a)) {
        if (stall && pair_shape(a)) return QKMLA_ERR_UNSUPPORTED;   // the hook exists in the 64-row kernel only
        plan->kernel = 1;
        plan->num_splits = a->num_splits;
        plan->parts = 0;
        plan->ws_bytes = tc_workspace(a, sms);
        return QKMLA_OK;
    }
    if (stall) return QKMLA_ERR_UNSUPPORTED;
    if (!(a->flags & QKMLA_FLAG_FORCE_SIMT) && q8_tc_supported(a, x) && tc_splits(a)) {
        plan->kernel = 1;
        plan->num_splits = a->num_splits;
        plan->parts = 0;
        plan->ws_bytes = q8_tc_workspace(a, sms);
        return QKMLA_OK;
    }
    plan->kernel = 0;
    int ns = a->num_splits;
    if (ns == 0) {
        const int64_t base = (int64_t)a->B * a->s_q * a->G;
        int64_t max_len = (int64_t)a->max_pages * a->page_size;
        if (x.window > 0) max_len = std::min(max_len, (int64_t)x.window + x.sinks);
        int64_t want = (2LL * sms + base - 1) / base;
        const int64_t cap = (max_len + 255) / 256;
        if (want > cap) want = cap;
        if (want < 1) want = 1;
        if (want > 256) want = 256;
        ns = (int)want;
    }
    plan->num_splits = ns;
    plan->parts = ns;
    const int64_t rows_h = (int64_t)a->B * a->s_q * a->H;
    plan->ws_bytes = ns > 1 ? (size_t)rows_h * ns * (a->d_c + 1) * sizeof(float) : 0;
    return QKMLA_OK;
}

}  // namespace qkmla

using namespace qkmla;

extern "C" {

int qkmla_version(void) { return 100; }

const char* qkmla_status_string(int st) {
    switch (st) {
        case QKMLA_OK: return "ok";
        case QKMLA_ERR_INVALID: return "invalid argument";
        case QKMLA_ERR_UNSUPPORTED: return "unsupported configuration";
        case QKMLA_ERR_CUDA: return "CUDA error";
        case QKMLA_ERR_WORKSPACE: return "workspace missing or too small";
        case QKMLA_ERR_DEVICE_BOUNDS: return "device-side bounds error (page id or sequence length)";
        case QKMLA_ERR_TIMEOUT: return "device-side bounded wait expired";
    }
    return "unknown status";
}

int qkmla_absorb_query(const float* q, const float* gamma_q, const float* gamma_k, const float* w_k, int rows,
                       int H, int G, int d_h, int d_c, float eps, unsigned flags, void* q_tilde, int qt_dtype,
                       float* alpha_q, void* stream) {
    const bool plain = (flags & QKMLA_FLAG_PLAIN_MLA) != 0;
    if (rows < 1 || H < 1 || G < 1 || d_h < 1 || d_c < 1 || H % G) return QKMLA_ERR_INVALID;
    if (d_h > 256 || d_c % 8) return QKMLA_ERR_INVALID;
    if (!q || !w_k || !q_tilde || !alpha_q) return QKMLA_ERR_INVALID;
    if (!plain && (!gamma_q || !gamma_k)) return QKMLA_ERR_INVALID;
    if (!(eps >= 0.f)) return QKMLA_ERR_INVALID;
    if (qt_dtype != QKMLA_F32 && qt_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    return launch_absorb(q, gamma_q, gamma_k, w_k, rows, H, G, d_h, d_c, eps, plain, q_tilde, qt_dtype, alpha_q,
                         (cudaStream_t)stream);
}

int qkmla_append(const float* c_new, const float* k_rope_new, const float* w_k, const float* gamma_rope_k,
                 const int64_t* slot_mapping, int N, int G, int d_c, int d_h, int d_r, float eps, unsigned flags,
                 void* kv_cache, int cache_dtype, void* ak_cache, int64_t num_slots, void* stream) {
    const bool plain = (flags & QKMLA_FLAG_PLAIN_MLA) != 0;
    if (N < 0 || G < 1 || d_c < 1 || d_h < 1 || d_r < 0 || num_slots < 1) return QKMLA_ERR_INVALID;
    if (d_h > 256) return QKMLA_ERR_INVALID;
    if (cache_dtype != QKMLA_F32 && cache_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    if (N == 0) return QKMLA_OK;
    if (!c_new || !w_k || !slot_mapping || !kv_cache || !ak_cache) return QKMLA_ERR_INVALID;
    if (d_r > 0 && !k_rope_new) return QKMLA_ERR_INVALID;
    if (!(eps >= 0.f)) return QKMLA_ERR_INVALID;
    const bool ak_f16 = !plain && (flags & QKMLA_FLAG_ALPHA_F16) != 0;
    return launch_append(c_new, k_rope_new, w_k, gamma_rope_k, slot_mapping, N, G, d_c, d_h, d_r, eps, plain,
                         kv_cache, cache_dtype, ak_cache, ak_f16, num_slots, nullptr, 0.f, (cudaStream_t)stream);
}

int qkmla_append_rope(const float* c_new, const float* k_rope_raw, const int32_t* positions, float rope_theta,
                      const float* w_k, const float* gamma_rope_k, const int64_t* slot_mapping, int N, int G, int d_c,
                      int d_h, int d_r, float eps, unsigned flags, void* kv_cache, int cache_dtype, void* ak_cache,
                      int64_t num_slots, void* stream) {
    if (N > 0 && d_r > 0 && (!positions || !(rope_theta > 1.f) || d_r % 2)) return QKMLA_ERR_INVALID;
    if (d_r > 64) return QKMLA_ERR_UNSUPPORTED;
    const bool plain = (flags & QKMLA_FLAG_PLAIN_MLA) != 0;
    if (N < 0 || G < 1 || d_c < 1 || d_h < 1 || d_r < 0 || num_slots < 1) return QKMLA_ERR_INVALID;
    if (d_h > 256) return QKMLA_ERR_INVALID;
    if (cache_dtype != QKMLA_F32 && cache_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    if (N == 0) return QKMLA_OK;
    if (!c_new || !w_k || !slot_mapping || !kv_cache || !ak_cache) return QKMLA_ERR_INVALID;
    if (d_r > 0 && !k_rope_raw) return QKMLA_ERR_INVALID;
    if (!(eps >= 0.f)) return QKMLA_ERR_INVALID;
    const bool ak_f16 = !plain && (flags & QKMLA_FLAG_ALPHA_F16) != 0;
    return launch_append(c_new, k_rope_raw, w_k, gamma_rope_k, slot_mapping, N, G, d_c, d_h, d_r, eps, plain,
                         kv_cache, cache_dtype, ak_cache, ak_f16, num_slots, d_r > 0 ? positions : nullptr,
                         rope_theta, (cudaStream_t)stream);
}

int qkmla_append_q8(const float* c_new, const float* k_rope_new, const int32_t* positions, float rope_theta,
                    const float* w_k, const float* gamma_rope_k, const int64_t* slot_mapping, int N, int G, int d_c,
                    int d_h, int d_r, float eps, unsigned flags, void* kv_cache, float* kv_scale, void* ak_cache,
                    int64_t num_slots, void* stream) {
    const bool plain = (flags & QKMLA_FLAG_PLAIN_MLA) != 0;
    if (N < 0 || G < 1 || G > 65535 || d_c < 1 || d_h < 1 || d_r < 0 || num_slots < 1) return QKMLA_ERR_INVALID;
    if (d_h > 256 || d_c % 2 || !(eps >= 0.f)) return QKMLA_ERR_INVALID;
    if (d_c > 512 || d_r > 64) return QKMLA_ERR_UNSUPPORTED;
    if (N == 0) return QKMLA_OK;
    if (positions && d_r > 0 && (!(rope_theta > 1.f) || d_r % 2)) return QKMLA_ERR_INVALID;
    if (!c_new || !w_k || !slot_mapping || !kv_cache || !kv_scale || !ak_cache) return QKMLA_ERR_INVALID;
    if (d_r > 0 && !k_rope_new) return QKMLA_ERR_INVALID;
    if (!aligned(kv_cache, 2) || !aligned(kv_scale, 4)) return QKMLA_ERR_INVALID;
    const bool ak_f16 = !plain && (flags & QKMLA_FLAG_ALPHA_F16) != 0;
    return launch_append_q8(c_new, k_rope_new, w_k, gamma_rope_k, slot_mapping, N, G, d_c, d_h, d_r, eps, plain,
                            (uint8_t*)kv_cache, kv_scale, ak_cache, ak_f16, num_slots, d_r > 0 ? positions : nullptr,
                            rope_theta, (cudaStream_t)stream);
}

}  // extern "C"

namespace {

size_t workspace_size(const qkmla_decode_args* a, const DecodeExt& x) {
    DecodePlan plan;
    if (plan_decode(a, x, &plan) != QKMLA_OK) return 0;
    return plan.ws_bytes;
}

const char* kernel_name(const qkmla_decode_args* a, const DecodeExt& x) {
    DecodePlan plan;
    if (plan_decode(a, x, &plan) != QKMLA_OK) return "invalid";
    return plan.kernel == 1 ? "tcgen05" : "simt";
}

int launch_count(const qkmla_decode_args* a, const DecodeExt& x) {
    DecodePlan plan;
    if (plan_decode(a, x, &plan) != QKMLA_OK) return 0;
    if (plan.kernel == 1)                                      // [scheduler,] decode[, combine]
        return (sched_in_kernel(a) ? 1 : 2) + (x.active() && never_splits(a, x) ? 0 : 1);
    return plan.parts > 1 ? 2 : 1;
}

int decode(const qkmla_decode_args* a, const DecodeExt& x, void* stream) {
    DecodePlan plan;
    const int rc = plan_decode(a, x, &plan);
    if (rc != QKMLA_OK) return rc;
    if (plan.ws_bytes > 0 && (!a->workspace || a->workspace_bytes < plan.ws_bytes)) return QKMLA_ERR_WORKSPACE;
    if (plan.ws_bytes > 0 && !aligned(a->workspace, 16)) return QKMLA_ERR_INVALID;
    if (plan.kernel == 1 && x.kv_scale) return launch_decode_q8(a, x, (cudaStream_t)stream);
    if (plan.kernel == 1) return launch_decode_tc(a, x, (cudaStream_t)stream);
    return launch_decode_simt(a, x, plan, (cudaStream_t)stream);
}

// The caller's extension as the library's; false for one the cache type cannot have.
bool read_ext(const qkmla_decode_args* a, const qkmla_decode_ext_args* e, DecodeExt* x) {
    *x = DecodeExt{};
    if (!a || !e) return false;
    x->kv_scale = e->kv_scale;
    // a window or sinks beyond the longest sequence mean all of it; kept below, no kernel's index can wrap
    const int64_t max_len = std::max<int64_t>(1, (int64_t)a->max_pages * a->page_size);
    x->window = (int)std::min<int64_t>(e->window, max_len);
    x->sinks = (int)std::min<int64_t>(e->sinks, max_len);
    return (a->cache_dtype == QKMLA_E4M3) == (e->kv_scale != nullptr);
}

}  // namespace

extern "C" {

size_t qkmla_decode_workspace_size(const qkmla_decode_args* a) { return workspace_size(a, DecodeExt{}); }

const char* qkmla_decode_kernel_name(const qkmla_decode_args* a) { return kernel_name(a, DecodeExt{}); }

int qkmla_decode_launch_count(const qkmla_decode_args* a) { return launch_count(a, DecodeExt{}); }

int qkmla_decode(const qkmla_decode_args* a, void* stream) { return decode(a, DecodeExt{}, stream); }

size_t qkmla_decode_ext_workspace_size(const qkmla_decode_args* a, const qkmla_decode_ext_args* e) {
    DecodeExt x;
    return read_ext(a, e, &x) ? workspace_size(a, x) : 0;
}

const char* qkmla_decode_ext_kernel_name(const qkmla_decode_args* a, const qkmla_decode_ext_args* e) {
    DecodeExt x;
    return read_ext(a, e, &x) ? kernel_name(a, x) : "invalid";
}

int qkmla_decode_ext_launch_count(const qkmla_decode_args* a, const qkmla_decode_ext_args* e) {
    DecodeExt x;
    return read_ext(a, e, &x) ? launch_count(a, x) : 0;
}

int qkmla_decode_ext(const qkmla_decode_args* a, const qkmla_decode_ext_args* e, void* stream) {
    DecodeExt x;
    return read_ext(a, e, &x) ? decode(a, x, stream) : QKMLA_ERR_INVALID;
}

int qkmla_get_device_status(void* stream) {
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return QKMLA_ERR_CUDA;
    int* p = device_status_ptr();
    if (!p) return QKMLA_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return QKMLA_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return QKMLA_ERR_CUDA;
    return v;
}

}  // extern "C"
