// qkmla_read_cache: rows of the paged cache read back into contiguous latents, RoPE keys and alpha^k.
//
// c[n] = cast(c^_t), c^_t the stored latent (8-bit cache: code x scale), r[n] = cast(k^rope_t), ak[n] =
// alpha^k_t, for row n of sequence b (out_start[b] <= n < out_start[b + 1]) and its token t = first[b] + n -
// out_start[b].  Every conversion is exact but the two to bf16 (fp32 cache; a code x scale below bf16's
// normal range), which round to nearest even.
//
// Bound: HBM, a row read and written once.  What costs time beyond that is the chain row -> sequence ->
// page -> slot in front of the row's own load, so a warp takes four neighbouring rows, its lanes follow the
// four chains at once, and the four rows' loads are all in flight together.  16-byte accesses (8 bytes of
// codes) where d_c, d_r and the bases allow, else element by element.
#include "common.cuh"

namespace qkmla {
namespace {

constexpr int kThreadsC = 256;
constexpr int kRowsW = 4;                  // rows a warp takes at once

struct ReadParams {
    const uint8_t* kv;
    const float* kv_scale;
    const void* ak;
    const int32_t* out_start;
    const int32_t* first;
    const int32_t* page_table;
    int64_t num_pages;
    void *c, *r;
    float* ak_out;
    int rows, B, d_c, d_r, G, page_size, max_pages, ak_f16;
    int* status;
};

// 8 elements of a row as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e4m3_to_float((uint8_t)((i < 4 ? u.x : u.y) >> (8 * (i & 3))));
    }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float one(const uint8_t* p) { return e4m3_to_float(*p); }

// The n elements at src[j] (times scale[j]) to dst + j * n, for the rows j whose bit is set.
template <typename T, typename OT, bool VEC>
__device__ __forceinline__ void copy_rows(const T* const (&src)[kRowsW], OT* dst, int n, const float (&scale)[kRowsW],
                                          unsigned rows, int lane) {
    if constexpr (VEC) {
        for (int e = lane * 8; e < n; e += 256) {
            float v[kRowsW][8];
#pragma unroll
            for (int j = 0; j < kRowsW; ++j)
                if (rows >> j & 1) load8(src[j] + e, v[j]);
#pragma unroll
            for (int j = 0; j < kRowsW; ++j)
                if (rows >> j & 1) {
                    if constexpr (sizeof(T) == 1) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[j][i] *= scale[j];
                    }
                    store8(dst + (int64_t)j * n + e, v[j]);
                }
        }
    } else {
        for (int j = 0; j < kRowsW; ++j)
            if (rows >> j & 1)
                for (int e = lane; e < n; e += 32) {
                    float v = one(src[j] + e);
                    if constexpr (sizeof(T) == 1) v *= scale[j];
                    Elem<OT>::store(dst + (int64_t)j * n + e, v);
                }
    }
}

// CT: the latent's stored type (uint8_t: e4m3 codes), RT: the RoPE key's.
template <typename CT, typename RT, typename OT, bool VEC>
__global__ void __launch_bounds__(kThreadsC) read_cache_kernel(const ReadParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t row0 = ((int64_t)blockIdx.x * (kThreadsC / 32) + (threadIdx.x >> 5)) * kRowsW;
    // lane j < 4 follows row row0 + j; its sequence by bisection of out_start (not written by the library)
    int64_t slot = -1;
    int b = 0;
    int64_t t = -1;
    const int64_t row = row0 + lane;
    if (lane < kRowsW && row < p.rows && row >= p.out_start[0] && row < p.out_start[p.B]) {
        int lo = 0, hi = p.B - 1;                        // the last b with out_start[b] <= row
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.out_start[mid] <= row) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        t = (p.first ? p.first[b] : 0) + (row - p.out_start[b]);
        if (t < 0 || t >= (int64_t)p.max_pages * p.page_size) {
            report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
            t = -1;
        }
    }
    if (t >= 0) slot = slot_of(p.page_table, b, (int)t, p.page_size, p.max_pages, p.num_pages, p.status);
    pdl_wait();
    pdl_trigger();
    const unsigned rows = __ballot_sync(0xffffffffu, slot >= 0);
    if (!rows) return;
    const int64_t row_bytes = (int64_t)p.d_c * sizeof(CT) + (int64_t)p.d_r * sizeof(RT);
    const CT* c[kRowsW];
    const RT* r[kRowsW];
    float scale[kRowsW];
    int64_t sl[kRowsW];
#pragma unroll
    for (int j = 0; j < kRowsW; ++j) {
        sl[j] = __shfl_sync(0xffffffffu, slot, j);
        if (sl[j] < 0) sl[j] = 0;
        const uint8_t* base = p.kv + sl[j] * row_bytes;
        c[j] = reinterpret_cast<const CT*>(base);
        r[j] = reinterpret_cast<const RT*>(base + (int64_t)p.d_c * sizeof(CT));
        scale[j] = sizeof(CT) == 1 ? p.kv_scale[sl[j]] : 1.f;
    }
    if (p.ak_out)
        for (int e = lane; e < kRowsW * p.G; e += 32) {
            const int j = e / p.G, g = e - j * p.G;
            int64_t s = sl[0];
#pragma unroll
            for (int q = 1; q < kRowsW; ++q) s = j == q ? sl[q] : s;
            if (rows >> j & 1)
                p.ak_out[(row0 + j) * p.G + g] = p.ak_f16 ? load_alpha<true>(p.ak, s * p.G + g) : load_alpha<false>(p.ak, s * p.G + g);
        }
    copy_rows<CT, OT, VEC>(c, reinterpret_cast<OT*>(p.c) + row0 * p.d_c, p.d_c, scale, rows, lane);
    if (p.d_r > 0) copy_rows<RT, OT, VEC>(r, reinterpret_cast<OT*>(p.r) + row0 * p.d_r, p.d_r, scale, rows, lane);
}

template <typename CT, typename RT, typename OT>
int launch_read(const ReadParams& p, bool vec, cudaStream_t s) {
    const int64_t per = kThreadsC / 32 * kRowsW;
    const dim3 grid((unsigned)((p.rows + per - 1) / per));
    const cudaError_t e = vec ? launch_pdl(read_cache_kernel<CT, RT, OT, true>, grid, dim3(kThreadsC), 0, s, p)
                              : launch_pdl(read_cache_kernel<CT, RT, OT, false>, grid, dim3(kThreadsC), 0, s, p);
    return e == cudaSuccess ? QKMLA_OK : QKMLA_ERR_CUDA;
}

template <typename OT>
int launch_read_out(const ReadParams& p, int cache_dtype, bool vec, cudaStream_t s) {
    if (cache_dtype == QKMLA_F32) return launch_read<float, float, OT>(p, vec, s);
    if (cache_dtype == QKMLA_BF16) return launch_read<__nv_bfloat16, __nv_bfloat16, OT>(p, vec, s);
    return launch_read<uint8_t, __nv_bfloat16, OT>(p, vec, s);
}

}  // namespace
}  // namespace qkmla

using namespace qkmla;

extern "C" int qkmla_read_cache(const qkmla_read_cache_args* a, void* stream) {
    if (!a || a->rows < 0 || a->B < 1 || a->d_c < 1 || a->d_r < 0 || a->G < 0) return QKMLA_ERR_INVALID;
    if (a->page_size < 1 || a->max_pages < 1 || a->num_slots < 1 || a->num_slots % a->page_size) return QKMLA_ERR_INVALID;
    if ((int64_t)a->max_pages * a->page_size > INT32_MAX - 4096) return QKMLA_ERR_INVALID;
    const bool q8 = a->cache_dtype == QKMLA_E4M3;
    if (q8 != (a->kv_scale != nullptr) || (q8 && a->d_c % 2)) return QKMLA_ERR_INVALID;
    if (a->cache_dtype != QKMLA_F32 && a->cache_dtype != QKMLA_BF16 && !q8) return QKMLA_ERR_UNSUPPORTED;
    if (a->out_dtype != QKMLA_F32 && a->out_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    if (a->rows == 0) return QKMLA_OK;
    if (!a->kv_cache || !a->out_start || !a->c || (a->d_r > 0 && !a->r)) return QKMLA_ERR_INVALID;
    if (a->ak && (!a->ak_cache || a->G < 1)) return QKMLA_ERR_INVALID;
    const size_t esz = a->cache_dtype == QKMLA_F32 ? 4 : 2, osz = a->out_dtype == QKMLA_F32 ? 4 : 2;
    const bool f16 = (a->flags & QKMLA_FLAG_ALPHA_F16) != 0;
    if ((uintptr_t)a->kv_cache % esz || (uintptr_t)a->kv_scale % 4 || (uintptr_t)a->ak_cache % (f16 ? 2 : 4) ||
        (uintptr_t)a->out_start % 4 || (uintptr_t)a->first % 4 || (uintptr_t)a->page_table % 4 || (uintptr_t)a->c % osz ||
        (uintptr_t)a->r % osz || (uintptr_t)a->ak % 4)
        return QKMLA_ERR_INVALID;
    ReadParams p = {};
    p.kv = (const uint8_t*)a->kv_cache;
    p.kv_scale = a->kv_scale;
    p.ak = a->ak_cache;
    p.out_start = a->out_start;
    p.first = a->first;
    p.page_table = a->page_table;
    p.num_pages = a->num_slots / a->page_size;
    p.c = a->c;
    p.r = a->r;
    p.ak_out = a->ak;
    p.rows = a->rows;
    p.B = a->B;
    p.d_c = a->d_c;
    p.d_r = a->d_r;
    p.G = a->G;
    p.page_size = a->page_size;
    p.max_pages = a->max_pages;
    p.ak_f16 = f16 ? 1 : 0;
    p.status = device_status_ptr();
    // a vector is 8 elements: 8 to 32 bytes, loaded and stored 16 (codes: 8) at a time
    const bool vec = a->d_c % 8 == 0 && a->d_r % 8 == 0 && (uintptr_t)a->kv_cache % 16 == 0 && (uintptr_t)a->c % 16 == 0 &&
                     (uintptr_t)a->r % 16 == 0 && (!q8 || (a->d_c % 16 == 0));
    cudaStream_t s = (cudaStream_t)stream;
    return a->out_dtype == QKMLA_F32 ? launch_read_out<float>(p, a->cache_dtype, vec, s)
                                     : launch_read_out<__nv_bfloat16>(p, a->cache_dtype, vec, s);
}
