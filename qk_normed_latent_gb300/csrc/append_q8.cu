// qkmla_append_q8 kernel: write new tokens into the 8-bit latent cache.
//
// A latent is stored as e4m3 codes x and one power-of-two scale s (c^ = s x);
// alpha^k_g = 1 / sqrt(mean_j (c^ W^K_g)_j^2 + eps) is the statistic of what is
// stored, so decode normalises exactly the keys it sees.
//
// Plain-load kernel: CTA (token tile, g) holds 32 tokens and one group.  It takes
// each token's scale from its largest magnitude, forms the keys (fp32, one fmaf
// chain per element over ascending k) chunk by chunk through shared memory and
// reduces them to their sum of squares; the g = 0 CTA also stores the codes, the
// scale and the RoPE key.
#include "common.cuh"
#include "rope.cuh"

namespace qkmla {

namespace {

constexpr int kTT = 32;        // tokens per CTA
constexpr int kKC = 64;        // d_c chunk staged per step
constexpr int kThreads = 256;
constexpr int kMaxJ = 8;       // d_h <= 256

__global__ void __launch_bounds__(kThreads)
append_q8_plain_kernel(const float* __restrict__ c_new, const float* __restrict__ r_new, const float* __restrict__ wk,
                       const float* __restrict__ grk, const int64_t* __restrict__ slots, int N, int G, int d_c,
                       int d_h, int d_r, float eps, int plain, uint8_t* __restrict__ kv, float* __restrict__ kv_scale,
                       void* __restrict__ ak, int ak_f16, int64_t num_slots, const int32_t* __restrict__ positions,
                       float theta, int* status) {
    __shared__ float Cs[kTT][kKC + 1];
    __shared__ float scale_s[kTT], inv_s[kTT];
    __shared__ RopeFreq freq[32];
    extern __shared__ float Ws[];              // [kKC][d_h]
    const int g = blockIdx.y;
    const int n0 = blockIdx.x * kTT;
    const int tid = threadIdx.x, tx = tid & 31, ty = tid >> 5;   // ty: 0..7
    const int nj = (d_h + 31) / 32;
    if (positions && tid < d_r / 2) freq[tid] = rope_freq(theta, tid, d_r);
    pdl_wait();
    pdl_trigger();
    for (int tl = ty; tl < kTT; tl += kThreads / 32) {
        float top = 0.f;
        if (n0 + tl < N)
            for (int k = tx; k < d_c; k += 32) top = fmaxf(top, fabsf(c_new[(int64_t)(n0 + tl) * d_c + k]));
        top = warp_max(top);
        if (tx == 0) scale_s[tl] = e4m3_scale(top, &inv_s[tl]);
    }

    float acc[4][kMaxJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kMaxJ; ++j) acc[i][j] = 0.f;

    const float* wg = wk + (int64_t)g * d_c * d_h;
    for (int k0 = 0; k0 < d_c; k0 += kKC) {
        __syncthreads();
        for (int e = tid; e < kTT * kKC; e += kThreads) {
            const int tl = e / kKC, k = e % kKC;
            const int n = n0 + tl;
            // the statistic is taken over the STORED latent
            Cs[tl][k] = (n < N && k0 + k < d_c)
                            ? e4m3_to_float(e4m3_code(c_new[(int64_t)n * d_c + k0 + k], inv_s[tl])) * scale_s[tl]
                            : 0.f;
        }
        for (int e = tid; e < kKC * d_h; e += kThreads) {
            const int k = e / d_h, j = e % d_h;
            Ws[k * d_h + j] = (k0 + k < d_c) ? wg[(int64_t)(k0 + k) * d_h + j] : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < kKC; ++k) {
            float a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = Cs[ty + 8 * i][k];
#pragma unroll
            for (int j = 0; j < kMaxJ; ++j) {
                if (j < nj) {
                    const int jj = tx + 32 * j;
                    const float b = (jj < d_h) ? Ws[k * d_h + jj] : 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i][j] = fmaf(a[i], b, acc[i][j]);
                }
            }
        }
    }

    // alpha^k_{t,g}: warp ty owns tokens ty + 8 i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < kMaxJ; ++j) ss = fmaf(acc[i][j], acc[i][j], ss);
        ss = warp_sum(ss);
        const int n = n0 + ty + 8 * i;
        if (tx == 0 && n < N) {
            const int64_t s = slots[n];
            if (s >= num_slots) {
                report(status, QKMLA_ERR_DEVICE_BOUNDS);
            } else if (s >= 0) {
                store_alpha(ak, s * G + g, plain ? 1.f : 1.f / sqrtf(ss / (float)d_h + eps), ak_f16 != 0);
            }
        }
    }

    if (g != 0) return;
    // codes, scale and the RoPE key (rotated, then normalised on its own), one warp per token
    for (int tl = ty; tl < kTT; tl += kThreads / 32) {
        const int n = n0 + tl;
        if (n >= N) break;
        const int64_t s = slots[n];
        if (s < 0 || s >= num_slots) continue;
        uint8_t* dst = kv + s * (int64_t)(d_c + 2 * d_r);
        for (int k = tx; k < d_c; k += 32) dst[k] = e4m3_code(c_new[(int64_t)n * d_c + k], inv_s[tl]);
        if (tx == 0) kv_scale[s] = scale_s[tl];
        float rv[2];                                  // d_r <= 64: elements tx and tx + 32
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = tx + 32 * u;
            rv[u] = j < d_r ? r_new[(int64_t)n * d_r + j] : 0.f;
            if (positions) {
                const float w = __shfl_xor_sync(0xffffffffu, rv[u], 1);
                if (j < d_r) {
                    float c, sn;
                    rope_cos_sin(positions[n], freq[j >> 1], &c, &sn);
                    rv[u] = rope_apply(j, rv[u], w, c, sn);
                }
            }
        }
        const float ss = warp_sum(fmaf(rv[0], rv[0], rv[1] * rv[1]));
        const float beta = plain ? 1.f : 1.f / sqrtf(ss / (float)d_r + eps);
        __nv_bfloat16* rope = reinterpret_cast<__nv_bfloat16*>(dst + d_c);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int j = tx + 32 * u;
            if (j < d_r) rope[j] = __float2bfloat16_rn(plain ? rv[u] : rv[u] * (grk ? grk[j] : 1.f) * beta);
        }
    }
}

}  // namespace

int launch_append_q8(const float* c_new, const float* r_new, const float* wk, const float* grk, const int64_t* slots,
                     int N, int G, int d_c, int d_h, int d_r, float eps, bool plain, uint8_t* kv, float* kv_scale,
                     void* ak, bool ak_f16, int64_t num_slots, const int32_t* positions, float rope_theta,
                     cudaStream_t s) {
    const size_t smem = (size_t)kKC * d_h * sizeof(float);
    if (cudaFuncSetAttribute(append_q8_plain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return QKMLA_ERR_CUDA;
    dim3 grid((N + kTT - 1) / kTT, G);
    return launch_pdl(append_q8_plain_kernel, grid, dim3(kThreads), smem, s, c_new, r_new, wk, grk, slots, N, G, d_c,
                      d_h, d_r, eps, (int)plain, kv, kv_scale, ak, (int)ak_f16, num_slots, positions, rope_theta,
                      device_status_ptr()) == cudaSuccess
               ? QKMLA_OK
               : QKMLA_ERR_CUDA;
}

}  // namespace qkmla
