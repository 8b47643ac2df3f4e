// Shared device helpers of the QK-Normed MLA decode library (sm_103a).
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "../../include/qkmla.h"

namespace qkmla {

// Record the first device-side error in the per-device status word `st`
// (read and cleared by qkmla_get_device_status()).
__device__ __forceinline__ void report(int* st, int code) {
    if (st) atomicCAS(st, 0, code);
}

// Programmatic dependent launch.  Every kernel of the library is launched with
// programmatic stream serialization: it may start while the previous kernel on
// the stream is still running, so it first does only work that touches no
// global memory, then waits (pdl_wait) until the previous grid has completed and
// its writes are visible, and then lets the next kernel start its own launch
// (pdl_trigger; a kernel that never does is waited for in full, as by a launch without
// the attribute).  Launched without the attribute, both are no-ops.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float load(const float* p) { return *p; }
    static __device__ __forceinline__ float cast(float x) { return x; }
    static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ float cast(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
};

// The 8-bit latent cache: a row is d_c e4m3 codes, then d_r bf16 RoPE values.
struct E4M3 {};

__device__ __forceinline__ float e4m3_to_float(uint8_t v) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

// Power-of-two scale of a latent with largest magnitude `top`: the least 2^e with
// top <= 448 2^e (448 = 0.875 2^9 is the largest e4m3 value), 0 for a zero latent.
// e4m3 is a floating-point format, so a power of two loses nothing against
// top / 448 but up to one binade of its 2^-9..448 range, and makes c / s, s x and
// every later product with s exact.
__device__ __forceinline__ float e4m3_scale(float top, float* inv) {
    if (!(top > 0.f)) { *inv = 0.f; return 0.f; }
    // top = 1.f x 2^(E - 127), so 2^(E - 135) <= top / 256 and one more binade above 1.75 2^(E - 127)
    const int b = __float_as_int(fminf(top, 3.402823466e38f));
    const int e = max((b >> 23) - 135 + ((b & 0x7fffff) > 0x600000 ? 1 : 0), -126);
    *inv = __int_as_float((127 - e) << 23);
    return __int_as_float((127 + e) << 23);
}
// Code of c with the scale 1 / inv; a value that is not finite becomes NaN.
__device__ __forceinline__ uint8_t e4m3_code(float c, float inv) {
    if (!isfinite(c)) return 0x7F;
    return (uint8_t)__nv_cvt_float_to_fp8(c * inv, __NV_SATFINITE, __NV_E4M3);
}

// Tokens a query of causal length n sees through a window with sinks: all of them
// (window 0, or nothing between the sinks and the window), else [0, sinks) and
// [n - window, n), numbered 0 .. count - 1 without the gap.
struct VisibleRange {
    int count, head, gap;
    __host__ __device__ __forceinline__ VisibleRange(int n, int window, int sinks) {
        const int first = n - window;
        const bool cut = window > 0 && first > sinks;
        head = cut ? sinks : n;
        gap = cut ? first - sinks : 0;
        count = n - gap;
    }
    __host__ __device__ __forceinline__ int token(int u) const { return u < head ? u : u + gap; }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Physical slot of token t of sequence b (see the cache convention in qkmla.h).
// Returns -1 (and records a bounds error) for a page id outside [0, num_pages).
__device__ __forceinline__ int64_t slot_of(const int32_t* page_table, int b, int t, int page_size,
                                           int max_pages, int64_t num_pages, int* st) {
    const int p = t / page_size;
    const int64_t page = page_table ? (int64_t)page_table[(int64_t)b * max_pages + p]
                                    : (int64_t)b * max_pages + p;
    if (page < 0 || page >= num_pages) {
        report(st, QKMLA_ERR_DEVICE_BOUNDS);
        return -1;
    }
    return page * page_size + (t % page_size);
}

// alpha^k entry `idx` of the A^k_cache, stored as fp32 or (f16) as its RNE half cast.
__device__ __forceinline__ void store_alpha(void* ak, int64_t idx, float v, bool f16) {
    if (f16) reinterpret_cast<__half*>(ak)[idx] = __float2half_rn(v);
    else reinterpret_cast<float*>(ak)[idx] = v;
}
template <bool F16>
__device__ __forceinline__ float load_alpha(const void* ak, int64_t idx) {
    if constexpr (F16) return __half2float(reinterpret_cast<const __half*>(ak)[idx]);
    else return reinterpret_cast<const float*>(ak)[idx];
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Host: launch `kernel` on `s` with programmatic stream serialization.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace qkmla

// Launch-side helpers (host).
namespace qkmla {
int launch_absorb(const float* q, const float* gq, const float* gk, const float* wk, int rows, int H,
                  int G, int d_h, int d_c, float eps, bool plain, void* qt, int qt_dtype, float* aq,
                  cudaStream_t s);
bool absorb_tc_supported(const float* q, const float* wk, int d_h, int d_c);
int launch_absorb_tc(const float* q, const float* gq, const float* gk, const float* wk, int rows, int H, int G,
                     int d_h, int d_c, float eps, bool plain, void* qt, int qt_dtype, float* aq, cudaStream_t s);
int launch_append(const float* c_new, const float* r_new, const float* wk, const float* grk,
                  const int64_t* slots, int N, int G, int d_c, int d_h, int d_r, float eps, bool plain,
                  void* kv, int cache_dtype, void* ak, bool ak_f16, int64_t num_slots, const int32_t* positions,
                  float rope_theta, cudaStream_t s);

struct DecodePlan {
    int kernel;            // 0 = simt, 1 = tcgen05
    int num_splits;        // simt: splits per sequence
    int parts;             // number of partial (o, lse) records in the workspace
    size_t ws_bytes;
};
// qkmla_decode_ext's additions (all zero for qkmla_decode).
struct DecodeExt {
    const float* kv_scale;
    int window, sinks;
    bool active() const { return kv_scale != nullptr || window > 0; }
};
int plan_decode(const qkmla_decode_args* a, const DecodeExt& x, DecodePlan* plan);
int launch_decode_simt(const qkmla_decode_args* a, const DecodeExt& x, const DecodePlan& plan, cudaStream_t s);
int launch_decode_tc(const qkmla_decode_args* a, const DecodeExt& x, cudaStream_t s);
bool tc_supported(const qkmla_decode_args* a);
bool pair_shape(const qkmla_decode_args* a);        // served by the two-CTA cluster kernel
bool sched_in_kernel(const qkmla_decode_args* a);   // split plan computed by the decode kernels themselves
size_t tc_workspace(const qkmla_decode_args* a, int sms);
bool q8_tc_supported(const qkmla_decode_args* a, const DecodeExt& x);   // 8-bit cache, tensor-core kernel
// qkmla_decode_ext calls whose arguments alone rule out a split sequence: no combine kernel.
bool never_splits(const qkmla_decode_args* a, const DecodeExt& x);
size_t q8_tc_workspace(const qkmla_decode_args* a, int sms);
int launch_decode_q8(const qkmla_decode_args* a, const DecodeExt& x, cudaStream_t s);
int launch_append_q8(const float* c_new, const float* r_new, const float* wk, const float* grk, const int64_t* slots,
                     int N, int G, int d_c, int d_h, int d_r, float eps, bool plain, uint8_t* kv, float* kv_scale,
                     void* ak, bool ak_f16, int64_t num_slots, const int32_t* positions, float rope_theta,
                     cudaStream_t s);
int launch_combine(const float* o_part, const float* lse_part, int rows, int nsplit, int d_c, void* o,
                   int o_dtype, float* lse, cudaStream_t s);
int device_sm_count();
int* device_status_ptr();   // this device's status word (lazily resolved), or nullptr
}  // namespace qkmla
