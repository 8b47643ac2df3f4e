// qkmla_read_cache: rows of the paged cache read back into contiguous latents, RoPE keys and alpha^k.
//
// c[n] = cast(c^_t), c^_t the stored latent (8-bit cache: code x scale), r[n] = cast(k^rope_t), ak[n] =
// alpha^k_t, for row n of sequence b (out_start[b] <= n < out_start[b + 1]) and its token t = first[b] + n -
// out_start[b].  Every conversion is exact but the two to bf16 (fp32 cache; a code x scale below bf16's
// normal range), which round to nearest even.
//
// Bound: HBM, a row read and written once.  What costs time beyond that is the chain row -> sequence ->
// page -> slot in front of the row's own load, so a warp takes four neighbouring rows, its lanes follow the
// four chains at once, and all that the four rows need -- latents, RoPE keys, scales, alpha^k -- is on its way
// before the first value is used.  32768 rows of an 8-bit cache (512 + 64) to bf16: 26.4 us with the rows one after
// the other, 11.7 so (61 MB: 5.2 TB/s); 38200 bf16 rows (256 + 32) of 16 sequences to fp32: 17.7 and 14.4, with
// whole sectors a store 13.4 us (67 MB: 5.0 TB/s).  Those are calls in a row that overlapped; since the next launch waits for the
// last store they are 12.6 and 14.7 apart.  16-byte accesses (8 bytes of codes) where d_c, d_r and the bases allow, else element by element.
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

// 8 elements of a row as they are stored, and as fp32.
template <typename T> struct Eight {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (sizeof(T) == 1) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x; w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                const uint4 u = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8], float scale) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
            else if constexpr (sizeof(T) == 2) v[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
            else v[i] = e4m3_to_float((uint8_t)(w[i >> 2] >> (8 * (i & 3)))) * scale;
        }
    }
};
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    if ((uintptr_t)p % 32 == 0) {                          // whole sectors at once (all of a row's pieces, or none)
        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
                     "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
        return;
    }
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
    pdl_wait();                                          // (no early launch of the next kernel: append reads new tokens ahead of its wait)
    const unsigned rows = __ballot_sync(0xffffffffu, slot >= 0);
    if (!rows) return;
    const int64_t row_bytes = (int64_t)p.d_c * sizeof(CT) + (int64_t)p.d_r * sizeof(RT);
    float my_scale = 1.f;
    if (sizeof(CT) == 1 && slot >= 0) my_scale = p.kv_scale[slot];       // lane j's row
    OT *out_c = reinterpret_cast<OT*>(p.c) + row0 * p.d_c, *out_r = reinterpret_cast<OT*>(p.r) + row0 * p.d_r;
    auto row_of = [&](int j) { return p.kv + max((int64_t)0, __shfl_sync(0xffffffffu, slot, j)) * row_bytes; };
    // the first 32 of the four rows' alpha^k
    float al = 0.f;
    const int aj = p.G > 0 ? lane / p.G : 4, ag = lane - aj * p.G;
    const int64_t a_slot = __shfl_sync(0xffffffffu, slot, aj & 3);
    const bool a_there = p.ak_out && aj < kRowsW && (rows >> (aj & 3) & 1);
    if (a_there) al = p.ak_f16 ? load_alpha<true>(p.ak, a_slot * p.G + ag) : load_alpha<false>(p.ak, a_slot * p.G + ag);
    if constexpr (VEC) {
        // RoPE keys: a vector a lane, first all rows' that 32 lanes hold
        const int rv = p.d_r / 8, rj = rv > 0 ? lane / rv : 4, re = (lane - rj * rv) * 8;
        const uint8_t* r_row = row_of(rj & 3);
        const bool r_there = rv > 0 && rj < kRowsW && (rows >> (rj & 3) & 1);
        Eight<RT> rope;
        if (r_there) rope.load(reinterpret_cast<const RT*>(r_row + (int64_t)p.d_c * sizeof(CT)) + re);
        constexpr int kStep = sizeof(CT) == 4 ? 256 : 512;   // latents of a row in flight
        for (int e0 = 0; e0 < p.d_c; e0 += kStep) {
            Eight<CT> x[kRowsW][kStep / 256];
#pragma unroll
            for (int j = 0; j < kRowsW; ++j) {
                const CT* c = reinterpret_cast<const CT*>(row_of(j));
#pragma unroll
                for (int q = 0; q < kStep / 256; ++q)
                    if ((rows >> j & 1) && e0 + q * 256 + lane * 8 < p.d_c) x[j][q].load(c + e0 + q * 256 + lane * 8);
            }
#pragma unroll
            for (int j = 0; j < kRowsW; ++j) {
                const float scale = __shfl_sync(0xffffffffu, my_scale, j);
#pragma unroll
                for (int q = 0; q < kStep / 256; ++q) {
                    const int e = e0 + q * 256 + lane * 8;
                    if ((rows >> j & 1) && e < p.d_c) {
                        float v[8];
                        x[j][q].get(v, scale);
                        store8(out_c + (int64_t)j * p.d_c + e, v);
                    }
                }
            }
        }
        if (r_there) {
            float v[8];
            rope.get(v, 1.f);
            store8(out_r + (int64_t)rj * p.d_r + re, v);
        }
        if (rv > 8)                                          // more than 32 vectors
            for (int j = 0; j < kRowsW; ++j) {
                const uint8_t* row = row_of(j);
                if (rows >> j & 1)
                    for (int e = lane * 8; e < p.d_r; e += 256) {
                        rope.load(reinterpret_cast<const RT*>(row + (int64_t)p.d_c * sizeof(CT)) + e);
                        float v[8];
                        rope.get(v, 1.f);
                        store8(out_r + (int64_t)j * p.d_r + e, v);
                    }
            }
    } else {
        for (int j = 0; j < kRowsW; ++j) {
            const uint8_t* row = row_of(j);
            const float scale = __shfl_sync(0xffffffffu, my_scale, j);
            if (!(rows >> j & 1)) continue;
            for (int e = lane; e < p.d_c; e += 32) {
                float v = one(reinterpret_cast<const CT*>(row) + e);
                if constexpr (sizeof(CT) == 1) v *= scale;
                Elem<OT>::store(out_c + (int64_t)j * p.d_c + e, v);
            }
            for (int e = lane; e < p.d_r; e += 32)
                Elem<OT>::store(out_r + (int64_t)j * p.d_r + e, one(reinterpret_cast<const RT*>(row + (int64_t)p.d_c * sizeof(CT)) + e));
        }
    }
    if (a_there) p.ak_out[(row0 + aj) * p.G + ag] = al;
    if (p.ak_out && p.G > 8)                                 // more than 32 of them
        for (int j = 0; j < kRowsW; ++j) {
            const int64_t sl = __shfl_sync(0xffffffffu, slot, j);
            if (rows >> j & 1)
                for (int g = lane; g < p.G; g += 32)
                    p.ak_out[(row0 + j) * p.G + g] = p.ak_f16 ? load_alpha<true>(p.ak, sl * p.G + g) : load_alpha<false>(p.ak, sl * p.G + g);
        }
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
