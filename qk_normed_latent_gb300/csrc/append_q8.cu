// qkmla_append_q8 kernel: write new tokens into the 8-bit latent cache.
//
// A latent is stored as e4m3 codes x and one power-of-two scale s (c^ = s x);
// alpha^k_g = 1 / sqrt(mean_j (c^ W^K_g)_j^2 + eps) is the statistic of what is
// stored, so decode normalises exactly the keys it sees.
//
// Tensor-core kernel (d_c 128 / 256 / 512, d_h 64 / 128).  The key statistic is a GEMM [N, d_c] x [d_c, d_h]
// per group whose result is only squared and summed.  The codes are exact in bf16; W^K is split into two
// bf16 parts, w = hi + lo up to 2^-17 of w, both columns of one B operand, so that one tcgen05.mma
// (M = 128 tokens, N = 2 d_h, K = 16) forms both products; the epilogue adds the parts, squares and sums a
// token's columns in one thread.  alpha^k is within ~1e-6 of the fp32 form, whose GEMM on the CUDA cores took
// 30 times as long.  A CTA owns up to 128 tokens: it quantises them once (scale, codes, and the codes' values
// as the A operand, all d_c columns in shared memory) and runs over its groups, W^K streaming through registers
// (a chunk of each loader set in flight) into a ring of 32-row chunks.  How many tokens and groups a CTA takes
// is chosen by the host (plan_q8): whole prompts want 128 tokens and all groups, so that a token is quantised
// once; a decode step has few tokens and spreads its groups over the GPU.
//
// Plain-load kernel (other dimensions): CTA (token tile, g) holds 32 tokens and one group.  It takes
// each token's scale from its largest magnitude, forms the keys (fp32, one fmaf
// chain per element over ascending k) chunk by chunk through shared memory and
// reduces them to their sum of squares; the g = 0 CTA also stores the codes, the
// scale and the RoPE key.
#include <algorithm>

#include "common.cuh"
#include "decode_common.cuh"
#include "rope.cuh"
#include "tc_ptx.cuh"

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

// ---------------------------------------------------------------------------
// tensor-core kernel
// ---------------------------------------------------------------------------
using namespace tc;
using dec::wait_bounded;

constexpr int kMT = 128;          // rows of the MMA: tokens of a CTA, at most
constexpr int kLoadWarps = 8;     // of a set; the sets take the chunks of W^K in turn (a set's chunk costs it
constexpr int kSets = 3;          // ~1000 cycles of dependent instructions, the MMAs 256)
constexpr int kEpiWarps = 4;
constexpr int kMmaWarp = kSets * kLoadWarps + kEpiWarps;
constexpr int kTcThreads = 32 * (kMmaWarp + 1);
constexpr int kChunk = 32;        // rows of W^K per ring stage
constexpr int kAhead = 1;         // chunks of a set in flight in registers

template <int DC, int DH>
struct AppendLayout {
    static constexpr int kN = 2 * DH;                          // hi and lo columns
    static constexpr int kA = DC / 64 * kMT * 128;             // bf16, K-major, 128-byte swizzle
    static constexpr int kStage = kChunk * kN * 2;             // bf16, MN-major: kN / 64 atoms of 64 columns
    static constexpr int kNst = 4;                              // divides the chunks of a group: slots are constants
    static constexpr int kOffMisc = kA + kNst * kStage;
    static constexpr int kBytes = kOffMisc + (2 * kNst + 5) * 8 + 16 + kMT * 4 + 1024;
    static_assert(DC / kChunk % kNst == 0 && kBytes <= 232448, "shared memory budget");
};

struct AppendQ8Params {
    const float *c_new, *r_new, *wk, *grk;
    const int64_t* slots;
    int N, G, d_r;
    float eps;
    int plain;
    uint8_t* kv;
    float* kv_scale;
    void* ak;
    int ak_f16;
    int64_t num_slots;
    const int32_t* positions;
    float theta;
    int tokens, groups;           // per CTA
    int* status;
};

// A read-only load that stays where it is written: as an ordinary one the compiler may move it down to its use.
__device__ __forceinline__ float4 load_stream(const float4* p) {
    float4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

template <int DC, int DH>
__global__ void __launch_bounds__(kTcThreads, 1) append_q8_tc_kernel(const AppendQ8Params p) {
    using LY = AppendLayout<DC, DH>;
    constexpr int NST = LY::kNst, kV = DC / 128, kF4 = kChunk * DH / 4 / (32 * kLoadWarps);
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint64_t* bfull = (uint64_t*)(sm + LY::kOffMisc);          // [NST] chunk written -> MMA (one arrive per warp)
    uint64_t* bempty = bfull + NST;                            // [NST] MMA done -> loaders
    uint64_t* dfull = bempty + NST;                            // [2] keys of a group done -> epilogue
    uint64_t* dfree = dfull + 2;                               // [2] read -> MMA
    uint64_t* drain = dfree + 2;
    uint32_t* tmem_slot = (uint32_t*)(drain + 1);
    float* scale_s = (float*)(tmem_slot + 4);
    __shared__ RopeFreq freq[32];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // warp: uniform
    const int n0 = blockIdx.x * p.tokens, n_tok = min(p.tokens, p.N - n0);
    const int g0 = blockIdx.y * p.groups, n_g = min(p.groups, p.G - g0);
    const int n_chunks = n_g * (DC / kChunk);
    // the CTAs start at different groups: together they would read the same few lines of W^K
    const int g_first = (int)blockIdx.x % n_g;
    auto group_at = [&](int gi) { return gi + g_first < n_g ? gi + g_first : gi + g_first - n_g; };

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&bfull[i], kLoadWarps);
            mbar_init(&bempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dfree[i], kEpiWarps);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (p.positions && tid < p.d_r / 2) freq[tid] = rope_freq(p.theta, tid, p.d_r);
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    // W^K: the loads of the first chunks go out before anything else (no kernel of the library writes it)
    const float4* w4 = reinterpret_cast<const float4*>(p.wk + (int64_t)g0 * DC * DH);
    const int set = warp / kLoadWarps, st = tid % (32 * kLoadWarps);   // loader set, thread in it
    float4 wv[kAhead][kF4];
    auto fetch = [&](int q, float4 (&v)[kF4]) {
#pragma unroll
        for (int i = 0; i < kF4; ++i)
            if (q < n_chunks)
                v[i] = load_stream(w4 + (int64_t)(group_at(q / (DC / kChunk)) * (DC / kChunk) + q % (DC / kChunk)) * (kChunk * DH / 4) +
                                   st + 32 * kLoadWarps * i);
    };
    if (warp < kSets * kLoadWarps) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) fetch(u * kSets + set, wv[u]);
    }
    __syncthreads();                                           // freq, barriers
    pdl_wait();                                                // the cache writes follow the previous kernel
    pdl_trigger();

    // ---- quantise: a warp per token, the next token's loads in flight ----
    constexpr int kQWarps = kMmaWarp;
    if (warp < kQWarps) {
        const bool store_cache = g0 == 0;
        float gr[2];                                           // d_r <= 64: elements lane and lane + 32
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int jj = lane + 32 * u;
            gr[u] = (jj < p.d_r && p.grk && !p.plain) ? p.grk[jj] : 1.f;
        }
        float4 v[kV];
        float rv[2];
        int64_t slot = -1;
        int pos = 0;
        auto load = [&](int tl) {
            const bool on = tl < n_tok;
            const float4* src = reinterpret_cast<const float4*>(p.c_new + (int64_t)(n0 + tl) * DC);
#pragma unroll
            for (int k = 0; k < kV; ++k)
                if (on) v[k] = load_stream(src + 32 * k + lane);
            slot = (on && store_cache) ? p.slots[n0 + tl] : -1;
            pos = (on && store_cache && p.positions) ? p.positions[n0 + tl] : 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int jj = lane + 32 * u;
                rv[u] = (on && store_cache && jj < p.d_r) ? p.r_new[(int64_t)(n0 + tl) * p.d_r + jj] : 0.f;
            }
        };
        load(warp);
        for (int tl = warp; tl < n_tok; tl += kQWarps) {
            float4 x4[kV];
            float r2[2] = {rv[0], rv[1]};
            const int64_t at = slot;
            const int turn = pos;
#pragma unroll
            for (int k = 0; k < kV; ++k) x4[k] = v[k];
            load(tl + kQWarps);
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < kV; ++k)
                top = fmaxf(top, fmaxf(fmaxf(fabsf(x4[k].x), fabsf(x4[k].y)), fmaxf(fabsf(x4[k].z), fabsf(x4[k].w))));
            top = warp_max(top);
            float inv;
            const float s = e4m3_scale(top, &inv);
            const bool store = at >= 0 && at < p.num_slots;
            uint8_t* row = p.kv + at * (int64_t)(DC + 2 * p.d_r);
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                float x[4] = {x4[k].x, x4[k].y, x4[k].z, x4[k].w};
                if (isinf(top)) {                              // an infinity is stored as NaN, not saturated
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[u] = isinf(x[u]) ? __int_as_float(0x7fffffff) : x[u];
                }
                const uint32_t c01 = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t c23 = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
                const float2 f01 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c01, __NV_E4M3)));
                const float2 f23 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c23, __NV_E4M3)));
                const __nv_bfloat162 b01 = __floats2bfloat162_rn(f01.x, f01.y), b23 = __floats2bfloat162_rn(f23.x, f23.y);
                const int col = 128 * k + 4 * lane;
                uint2 w;
                w.x = *reinterpret_cast<const uint32_t*>(&b01);
                w.y = *reinterpret_cast<const uint32_t*>(&b23);
                *reinterpret_cast<uint2*>(sm + (col >> 6) * (kMT * 128) + sw128_offset(tl, col & 63)) = w;
                if (store) *reinterpret_cast<uint32_t*>(row + col) = c01 | (c23 << 16);
            }
            if (lane == 0) {
                scale_s[tl] = s;
                if (store) p.kv_scale[at] = s;
                if (at >= p.num_slots) report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
            }
            if (store_cache) {                                 // the RoPE key: rotated, then normalised on its own
                if (p.positions) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int jj = lane + 32 * u;
                        const float w = __shfl_xor_sync(0xffffffffu, r2[u], 1);
                        if (jj < p.d_r) {
                            float c, sn;
                            rope_cos_sin(turn, freq[jj >> 1], &c, &sn);
                            r2[u] = rope_apply(jj, r2[u], w, c, sn);
                        }
                    }
                }
                const float ss = warp_sum(fmaf(r2[0], r2[0], r2[1] * r2[1]));
                const float beta = p.plain ? 1.f : 1.f / sqrtf(ss / (float)p.d_r + p.eps);
                __nv_bfloat16* rope = reinterpret_cast<__nv_bfloat16*>(row + DC);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int jj = lane + 32 * u;
                    if (store && jj < p.d_r) rope[jj] = __float2bfloat16_rn(r2[u] * gr[u] * beta);
                }
            }
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < kSets * kLoadWarps) {
        // ===================== W^K chunks: fp32 registers -> hi and lo bf16 =====================
        bool ok = true;
        for (int q0 = set; q0 < n_chunks && ok; q0 += kAhead * kSets) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int q = q0 + u * kSets;
                if (q >= n_chunks) break;
                const int s = q % NST;
                if (q >= NST) ok = __all_sync(0xffffffffu, wait_bounded(&bempty[s], ((q / NST) - 1) & 1, p.status));
                if (!ok) break;
                uint8_t* stg = sm + LY::kA + s * LY::kStage;
#pragma unroll
                for (int i = 0; i < kF4; ++i) {
                    const int f = st + 32 * kLoadWarps * i;
                    const int k = f / (DH / 4), jc = 4 * (f % (DH / 4));
                    const float4 w = wv[u][i];
                    const __nv_bfloat162 h01 = __floats2bfloat162_rn(w.x, w.y), h23 = __floats2bfloat162_rn(w.z, w.w);
                    const float2 r01 = __bfloat1622float2(h01), r23 = __bfloat1622float2(h23);
                    const __nv_bfloat162 l01 = __floats2bfloat162_rn(w.x - r01.x, w.y - r01.y);
                    const __nv_bfloat162 l23 = __floats2bfloat162_rn(w.z - r23.x, w.w - r23.y);
                    uint2 hv, lv;
                    hv.x = *reinterpret_cast<const uint32_t*>(&h01); hv.y = *reinterpret_cast<const uint32_t*>(&h23);
                    lv.x = *reinterpret_cast<const uint32_t*>(&l01); lv.y = *reinterpret_cast<const uint32_t*>(&l23);
                    // atom of 64 columns x 8 rows: 1024 bytes, the atom's 8-row groups back to back
                    uint8_t* dst = stg + (jc >> 6) * (kChunk * 128) + (k >> 3) * 1024 + (k & 7) * 128 +
                                   ((((jc & 63) >> 3) ^ (k & 7)) << 4) + (jc & 4) * 2;
                    *reinterpret_cast<uint2*>(dst) = hv;
                    *reinterpret_cast<uint2*>(dst + DH / 64 * (kChunk * 128)) = lv;
                }
                // the fence to the async proxy is the MMA thread's: here it would wait for the loads in flight
                __syncwarp();
                if (lane == 0) mbar_arrive(&bfull[s]);
                fetch(q + kAhead * kSets, wv[u]);
            }
        }
    } else if (warp == kMmaWarp) {
        // ===================== MMA issuer (uniform control flow, one lane's instructions) =====================
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const int groups = __shfl_sync(0xffffffffu, n_g, 0);
        const uint32_t id = idesc_bf16(kMT, LY::kN, 0, 1);
        const uint64_t a0 = smem_desc(smem_u32(sm), 16, 1024, kSwizzle128B);
        const uint64_t b0 = smem_desc(smem_u32(sm + LY::kA), kChunk * 128, 1024, kSwizzle128B);
        bool ok = true;
        uint32_t phase = 0;
        for (int gi = 0; gi < groups && ok; ++gi) {
            const uint32_t d = tm + (uint32_t)(gi & 1) * 256u;
            bool got = true;
            if (gi >= 2) got = wait_bounded(&dfree[gi & 1], ((gi >> 1) - 1) & 1, p.status);
            for (int c4 = 0; c4 < DC / kChunk; c4 += NST, phase ^= 1) {
#pragma unroll
                for (int s = 0; s < NST; s += 2) {             // two chunks a fence
                    got = got && wait_bounded(&bfull[s], phase, p.status) && wait_bounded(&bfull[s + 1], phase, p.status);
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                    fence_proxy_async_smem();                  // the loaders' writes, seen through the barriers
                    tc_fence_after();
                    const uint64_t a = a0 + (uint64_t)(((c4 + s) >> 1) * (kMT * 128 >> 4));
                    if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 2 * kChunk / 16; ++kk) {
                        mma_bf16(d, a + (uint64_t)(kk * 2),
                                    b0 + (uint64_t)(((s + (kk >> 1)) * LY::kStage + (kk & 1) * 2048) >> 4), id,
                                    (c4 > 0 || s > 0 || kk > 0) ? 1u : 0u);
                        if (kk & 1) mma_commit(&bempty[s + (kk >> 1)]);
                    }
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            if (ok && elect_one()) mma_commit(&dfull[gi & 1]);
            __syncwarp();
        }
        if (elect_one()) mma_commit(drain);
        __syncwarp();                            // no exit with an MMA in flight
        wait_bounded(drain, 0, p.status);
    } else {
        // ===================== epilogue: thread = token =====================
        const int sub = warp & 3, tl = 32 * sub + lane;
        const uint32_t lane_base = (uint32_t)(32 * sub) << 16;
        const bool on = tl < n_tok;
        const int64_t slot = on ? p.slots[n0 + tl] : -1;
        const float s = on ? scale_s[tl] : 0.f;
        for (int gi = 0; gi < n_g; ++gi) {
            const bool got = __all_sync(0xffffffffu, wait_bounded(&dfull[gi & 1], (gi >> 1) & 1, p.status));
            if (!got) break;
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(gi & 1) * 256u + lane_base;
            float ss[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int c = 0; c < DH; c += 16) {
                uint32_t h[16], l[16];
                tmem_ld16(d + c, h);
                tmem_ld16(d + DH + c, l);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const float k = __uint_as_float(h[u]) + __uint_as_float(l[u]);
                    ss[u & 3] = fmaf(k, k, ss[u & 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dfree[gi & 1]);
            const float mean = ((ss[0] + ss[1]) + (ss[2] + ss[3])) / (float)DH;   // of the keys of the codes
            if (slot >= 0 && slot < p.num_slots)
                store_alpha(p.ak, slot * p.G + g0 + group_at(gi), p.plain ? 1.f : 1.f / sqrtf(s * s * mean + p.eps), p.ak_f16 != 0);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Tokens and groups per CTA: the cheapest of a few splits by a simple model -- a fixed part, a part per token
// (quantising: a warp per token) and a part per group (its W^K streamed and multiplied), times the waves.
void plan_q8(int N, int G, int d_c, int d_h, int sms, int* tokens, int* groups) {
    const float per_token = 0.02f, per_group = 2.2f * (float)d_c * d_h / (512 * 128), fixed = 4.f;   // us
    float best = 1e30f;
    for (int t = 16; t <= kMT; t *= 2)
        for (int g = 1; g <= G; ++g) {
            const int64_t ctas = (int64_t)((N + t - 1) / t) * ((G + g - 1) / g);
            const float cost = (float)((ctas + sms - 1) / sms) * (fixed + per_token * t + per_group * g);
            if (cost < best) { best = cost; *tokens = t; *groups = g; }
        }
}

template <int DC, int DH>
cudaError_t launch_tc(const AppendQ8Params& p, cudaStream_t s) {
    auto k = append_q8_tc_kernel<DC, DH>;
    constexpr int bytes = AppendLayout<DC, DH>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((p.N + p.tokens - 1) / p.tokens, (p.G + p.groups - 1) / p.groups);
    return launch_pdl(k, grid, dim3(kTcThreads), bytes, s, p);
}

}  // namespace

int launch_append_q8(const float* c_new, const float* r_new, const float* wk, const float* grk, const int64_t* slots,
                     int N, int G, int d_c, int d_h, int d_r, float eps, bool plain, uint8_t* kv, float* kv_scale,
                     void* ak, bool ak_f16, int64_t num_slots, const int32_t* positions, float rope_theta,
                     cudaStream_t s) {
    const bool tc = (d_c == 128 || d_c == 256 || d_c == 512) && (d_h == 64 || d_h == 128) && d_r % 2 == 0 &&
                    ((uintptr_t)c_new % 16) == 0 && ((uintptr_t)wk % 16) == 0 && ((uintptr_t)kv % 4) == 0;
    if (tc) {
        const int sms = device_sm_count();
        if (sms <= 0) return QKMLA_ERR_CUDA;
        AppendQ8Params p{c_new, r_new, wk, grk, slots, N, G, d_r, eps, (int)plain, kv, kv_scale, ak, (int)ak_f16,
                         num_slots, positions, rope_theta, 0, 0, device_status_ptr()};
        plan_q8(N, G, d_c, d_h, sms, &p.tokens, &p.groups);
        const bool wide = d_h == 128;
        const cudaError_t e = d_c == 512   ? (wide ? launch_tc<512, 128>(p, s) : launch_tc<512, 64>(p, s))
                              : d_c == 256 ? (wide ? launch_tc<256, 128>(p, s) : launch_tc<256, 64>(p, s))
                                           : (wide ? launch_tc<128, 128>(p, s) : launch_tc<128, 64>(p, s));
        return e == cudaSuccess ? QKMLA_OK : QKMLA_ERR_CUDA;
    }
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
