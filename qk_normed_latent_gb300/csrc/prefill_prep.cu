// qkmla_prefill, the kernels ahead of the attention, and the packing of its weights.
//
// prefill_pack_kernel   W^K (fp32) and W^V (bf16) as fp16 K-major blocks, each matrix times a power of two
//                       that brings its largest value into [1, 2): fp16's 11 bits hold W^V's 8 exactly and
//                       W^K to 2^-11, whatever the weights' scale.
// prefill_query_kernel  q^ = q gamma_q gamma_k / rms(q) and the RoPE part likewise, one row (query token,
//                       head) a warp, times a power of two a row that brings its largest value into
//                       [1, 2), rounded to fp16; softmax_scale, log2 e and that power are the row's factor
//                       in the attention kernel, where it costs nothing.  HBM-bound: 768 bytes read and 384
//                       written a row.  Block 0 makes the plan instead.
// prefill_expand_kernel keys and values of 128 cached tokens, on the tensor cores.
#include "prefill.cuh"

namespace qkmla {
namespace pf {
namespace {

using namespace tc;

// ---------------------------------------------------------------------------
// weights
// ---------------------------------------------------------------------------
// Block (x, y): 64 latents (y) of one matrix (x: the G of W^K, then the G_v of W^V).
__global__ void __launch_bounds__(256) prefill_pack_kernel(const float* __restrict__ wk, const __nv_bfloat16* __restrict__ wv, int G,
                                                           int Gv, int d_c, int d_h, int d_v, uint8_t* __restrict__ packed) {
    const int m = blockIdx.x;
    const bool key = m < G;
    const int d = key ? d_h : d_v;
    const size_t n = (size_t)d_c * d;
    const float* k = wk + (size_t)m * n;
    const __nv_bfloat16* v = wv + (size_t)(key ? 0 : m - G) * n;
    __shared__ float tops[8];
    float top = 0.f;
    for (size_t i = threadIdx.x; i < n; i += 256) {
        const float a = fabsf(key ? k[i] : __bfloat162float(v[i]));
        if (isfinite(a)) top = fmaxf(top, a);
    }
    top = warp_max(top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, tops[i]);
    const int e = top > 0.f ? max(ilogbf(top), -126) : 0;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0 && blockIdx.y == 0) reinterpret_cast<int*>(packed)[m] = e;
    uint8_t* blocks = packed + kWeightTable;
    const int c0 = blockIdx.y * 64;
    const int first = key ? m * (d_h / 64) : G * (d_h / 64) + (m - G) * (d_v / 64);
    for (int i = threadIdx.x; i < 64 * d; i += 256) {
        const int c = i / d, j = i % d;                    // latent c0 + c, output column j
        const size_t at = (size_t)(c0 + c) * d + j;
        const float w = ldexpf(key ? k[at] : __bfloat162float(v[at]), -e);
        const int cb = first + j / 64;                     // 64-column block
        uint8_t* blk = blocks + ((size_t)(cb / 2) * (d_c / 64) + blockIdx.y) * kBlock;
        *reinterpret_cast<__half*>(blk + sw128_offset((cb & 1) * 64 + j % 64, c)) = __float2half_rn(w);
    }
}

// ---------------------------------------------------------------------------
// queries and the plan
// ---------------------------------------------------------------------------
constexpr int kThreadsQ = 256;
constexpr int kRowsWarp = 4;               // rows a warp has in flight

// Sum of the block's values ahead of this thread's; the whole sum in *all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warps, int64_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    int64_t ahead = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kThreadsQ / 32; ++i) {
        if (i < warp) ahead += warps[i];
        sum += warps[i];
    }
    *all = sum;
    return ahead + s - v;
}

__device__ void make_plan(const Params& p) {
    __shared__ int64_t warps[kThreadsQ / 32];
    const int tid = threadIdx.x;
    // sequences: lengths, first tiles, rows
    int64_t tiles = 0, tokens = 0, all;
    const int per = (p.B + kThreadsQ - 1) / kThreadsQ;
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b >= p.B) break;
        const int len = p.seq_lens[b];
        if (len < 0 || len > (int64_t)p.max_pages * p.page_size) continue;
        tiles += (len + kTile - 1) / kTile;
        tokens += len;
    }
    int64_t at = block_scan(tiles, warps, &all);
    int64_t sum;
    block_scan(tokens, warps, &sum);
    if (tid == 0 && sum > p.total_tokens) report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b >= p.B) break;
        int len = p.seq_lens[b];
        const int r0 = p.chunk_start[b], r1 = p.chunk_start[b + 1];
        bool ok = len >= 0 && len <= (int64_t)p.max_pages * p.page_size;
        const int64_t n = ok ? (len + kTile - 1) / kTile : 0;
        bool rows_ok = r0 >= 0 && r0 <= r1 && r1 <= p.rows && (b > 0 || r0 == 0);
        if (!ok || !rows_ok) report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
        const bool fits = at + n <= p.max_tiles;           // no tile is written beyond the workspace
        p.seq[b] = make_int4(ok && fits ? len : 0, (int)min(at, (int64_t)p.max_tiles), rows_ok ? r0 : 0, rows_ok ? r1 - r0 : 0);
        at += n;
    }
    for (int j = tid; j < p.nq; j += kThreadsQ) p.qinfo[2 * j] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    // query tiles: the tiles of tokens that any of their queries sees
    for (int b = tid >> 5; b < p.B; b += kThreadsQ / 32) {
        const int4 s = p.seq[b];
        const int n = s.w, j0 = first_slot(s.z, b, p.tq);
        for (int k = tid & 31; k * (int64_t)p.tq < n; k += 32) {
            const int i0 = k * p.tq, i1 = min(n, i0 + p.tq);
            const int lo = s.x - n + i0 + 1, hi = s.x - n + i1;        // causal lengths of the first and the last query
            const int total = hi > 0 ? (hi + kTile - 1) / kTile : 0;
            int head = total, gap = 0;
            if (p.window > 0 && lo - p.window > 0) {
                const int from = min((lo - p.window) / kTile, total);
                const int h = (min(p.sinks, lo - p.window) + kTile - 1) / kTile;
                if (from > h) { head = h; gap = from - h; }
            }
            p.qinfo[2 * (j0 + k)] = make_int4(b, i0, total - gap, head);
            p.qinfo[2 * (j0 + k) + 1] = make_int4(gap, lo, i1 - i0, 0);
        }
    }
    __syncthreads();
    const int pq = (p.nq + kThreadsQ - 1) / kThreadsQ;
    int64_t mine = 0;
    for (int k = 0; k < pq; ++k) {
        const int j = tid * pq + k;
        if (j >= p.nq) break;
        const int4 q = p.qinfo[2 * j];
        if (q.x >= 0) mine += q.z + kCostStart;
    }
    int64_t ahead = block_scan(mine, warps, &all);
    for (int k = 0; k < pq; ++k) {
        const int j = tid * pq + k;
        if (j >= p.nq) break;
        p.pre[j] = ahead;
        const int4 q = p.qinfo[2 * j];
        if (q.x >= 0) ahead += q.z + kCostStart;
    }
    if (tid == 0) p.pre[p.nq] = all;
}

template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (N == 4) { const float4 f = *reinterpret_cast<const float4*>(p); v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w; }
        else if constexpr (N == 2) { const float2 f = *reinterpret_cast<const float2*>(p); v[0] = f.x; v[1] = f.y; }
        else v[0] = *p;
    } else {
        uint32_t w[(N + 1) / 2];
        if constexpr (N == 4) { const uint2 u = *reinterpret_cast<const uint2*>(p); w[0] = u.x; w[1] = u.y; }
        else if constexpr (N == 2) w[0] = *reinterpret_cast<const uint32_t*>(p);
        else w[0] = *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
}
template <int N>
__device__ __forceinline__ void store_n(uint8_t* p, const float (&v)[N]) {
    if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
    else if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = pack_f16(v[0], v[1]);
    else *reinterpret_cast<__half*>(p) = __float2half_rn(v[0]);
}

// DH values of content and DR of RoPE a row; a lane holds DH / 32 and DR / 32 neighbours.
template <typename T, int DH, int DR>
__global__ void __launch_bounds__(kThreadsQ) prefill_query_kernel(const Params p) {
    constexpr int NH = DH / 32, NR = DR / 32, KU = DH / 64 + 1;
    pdl_wait();                                            // the workspace may still be in use
    pdl_trigger();
    if (blockIdx.x == 0) {
        make_plan(p);
        return;
    }
    const int lane = threadIdx.x & 31;
    float gam[NH], gr[NR];
#pragma unroll
    for (int i = 0; i < NH; ++i) gam[i] = p.gamma_q[lane * NH + i] * p.gamma_k[lane * NH + i];
#pragma unroll
    for (int i = 0; i < NR; ++i) gr[i] = p.gamma_rope ? p.gamma_rope[lane * NR + i] : 1.f;
    const int64_t item0 = ((int64_t)(blockIdx.x - 1) * (kThreadsQ / 32) + (threadIdx.x >> 5)) * kRowsWarp;
    const int64_t items = (int64_t)p.rows * p.H;
    // lane j < kRowsWarp finds the place of row item0 + j: its sequence by bisection
    int64_t dst = -1, tile = 0;
    int row = 0, r = 0, h = 0;
    if (lane < kRowsWarp && item0 + lane < items) {
        r = (int)((item0 + lane) / p.H);
        h = (int)((item0 + lane) % p.H);
        if (r >= p.chunk_start[0] && r < p.chunk_start[p.B]) {
            int lo = 0, hi = p.B - 1;                      // the last b with chunk_start[b] <= r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.chunk_start[mid] <= r) lo = mid;
                else hi = mid - 1;
            }
            const int cs = p.chunk_start[lo], i = r - cs;
            const int j = first_slot(cs, lo, p.tq) + i / p.tq;
            if (cs >= 0 && j < p.nq) {
                tile = (int64_t)(h / p.hp) * p.nq + j;
                row = (i % p.tq) * p.hp + h % p.hp;
                dst = (tile * 2 + (row >> 7)) * (KU * (int64_t)kBlock);
            }
        }
    }
    int64_t to[kRowsWarp];
    float x[kRowsWarp][NH], y[kRowsWarp][NR];
#pragma unroll
    for (int j = 0; j < kRowsWarp; ++j) {
        to[j] = __shfl_sync(0xffffffffu, dst, j);
        const int rr = __shfl_sync(0xffffffffu, r, j), hh = __shfl_sync(0xffffffffu, h, j);
        if (to[j] < 0) continue;
        load_n<T, NH>((const T*)p.q + rr * p.q_row + hh * p.q_head + lane * NH, x[j]);
        load_n<T, NR>((const T*)p.q_rope + rr * p.qr_row + hh * p.qr_head + lane * NR, y[j]);
    }
#pragma unroll
    for (int j = 0; j < kRowsWarp; ++j) {
        if (to[j] < 0) continue;
        float sx = 0.f, sy = 0.f;
#pragma unroll
        for (int i = 0; i < NH; ++i) sx = fmaf(x[j][i], x[j][i], sx);
#pragma unroll
        for (int i = 0; i < NR; ++i) sy = fmaf(y[j][i], y[j][i], sy);
        sx = warp_sum(sx);
        sy = warp_sum(sy);
        const float ax = 1.f / sqrtf(sx / DH + p.eps), ay = 1.f / sqrtf(sy / DR + p.eps);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NH; ++i) top = fmaxf(top, fabsf(x[j][i] = x[j][i] * ax * gam[i]));
#pragma unroll
        for (int i = 0; i < NR; ++i) top = fmaxf(top, fabsf(y[j][i] = y[j][i] * ay * gr[i]));
        top = warp_max(top);
        const int e = top > 0.f && isfinite(top) ? min(max(ilogbf(top), -100), 100) : 0;
        const float f = pow2i(-e);
#pragma unroll
        for (int i = 0; i < NH; ++i) x[j][i] *= f;
#pragma unroll
        for (int i = 0; i < NR; ++i) y[j][i] *= f;
        const int rw = __shfl_sync(0xffffffffu, row, j), r7 = rw & 127;
        const int64_t tl = __shfl_sync(0xffffffffu, tile, j);
        uint8_t* q = p.qt + to[j];
        const int col = lane * NH;
        store_n<NH>(q + (col >> 6) * kBlock + sw128_offset(r7, col & 63), x[j]);
        store_n<NR>(q + (KU - 1) * kBlock + sw128_offset(r7, lane * NR), y[j]);
        if (lane == 0) p.qc[tl * kRowsQ + rw] = p.scale_log2 * pow2i(e);
    }
}

// ---------------------------------------------------------------------------
// keys and values
// ---------------------------------------------------------------------------
// C [128 tokens, d_c] x [W^K_0 .. W^K_{G-1} | W^V_0 ..] in N-tiles of 128 columns.  The latents lie in shared
// memory for the whole CTA (d_c / 64 blocks), each token times a power of two of its own that brings its
// largest value into [1, 2): exact as fp16 for a bf16 or an 8-bit latent, but for what lies 2^-14 below that
// value.  Warps 0-7 gather and convert them, then take the results out of TMEM: a key row is scaled by the
// stored alpha^k, a value row by its share of the tile's common exponent.  Warp 8 streams the packed
// weights through a ring of blocks, warp 9 issues the products (M = N = 128, K = 64 a block), the
// accumulator double-buffered.  Blocks of results are staged in shared memory and leave as bulk copies.
//
// Bound: the tensor core for many tokens (2 d_c flops a value), next to it the weights, which every CTA
// streams through L2 (128 bytes a 256 flops: 63 bytes a cycle and SM at full rate).
constexpr int kThreadsE = 320;
constexpr int kRing = 4;                   // weight blocks in flight

struct ExpandLayout {
    int a, ring, stage, misc, bytes;
    __host__ __device__ explicit ExpandLayout(int d_c) {
        a = 0;
        ring = d_c / 64 * kBlock;
        stage = ring + kRing * kBlock;
        misc = stage + 2 * kBlock;
        bytes = misc + 2048 + 1024;
    }
};

template <bool Q8>
__global__ void __launch_bounds__(kThreadsE, 1) prefill_expand_kernel(const Params p, int splits) {
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    const ExpandLayout L(p.d_c);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.misc);          // [kRing]
    uint64_t* empty = full + kRing;                                     // [kRing]
    uint64_t* acc_full = empty + kRing;                                 // [2]
    uint64_t* acc_empty = acc_full + 2;                                 // [2]
    uint64_t* done = acc_empty + 2;
    int64_t* slots = reinterpret_cast<int64_t*>(done + 1);              // [128] slot of a token, -1 for none
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(slots + kTile);
    int* fail = reinterpret_cast<int*>(tmem_slot + 1);
    int* issued_s = fail + 1;
    int* warp_hi = issued_s + 1;                                        // [8]
    int* warp_lo = warp_hi + 8;                                         // [8]
    int* exps = warp_lo + 8;                                            // [128] exponent, or kNone / kBad
    constexpr int kNone = -1000, kBad = 1000;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = blockIdx.x / splits, part = blockIdx.x % splits;
    const int nkb = p.d_h / 64, nvb = p.d_v / 64, kb = p.d_c / 64;
    const int blocks = column_blocks(p.G, p.Gv, p.d_h, p.d_v), nt = (blocks + 1) / 2;
    const int n0 = nt * part / splits, n1 = nt * (part + 1) / splits;

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 256); }
        mbar_init(done, 1);
        *fail = 0;
        *issued_s = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    // the tile's sequence: the last one that starts at or before it and has tiles (uniform)
    int b = 0;
    {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.seq[mid].y <= tile) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
    }
    const int4 seq = p.seq[b];
    const int t0 = (tile - seq.y) * kTile;
    const int tokens = min(kTile, seq.x - t0);
    // tiles that no query of the step sees are left out
    bool wanted = tile >= seq.y && tokens > 0 && seq.w > 0;
    if (wanted && p.window > 0) {
        const int lo = seq.x - seq.w + 1 - p.window;                    // the first query's window starts here
        wanted = t0 < p.sinks || t0 + kTile > lo;
    }
    if (!wanted) {                                                      // uniform
        __syncthreads();
        if (warp == 9) tmem_dealloc(tmem, 256);
        return;
    }

    if (warp < 8) {
        // ---- gather: a warp's 16 tokens, their slots by its first 16 lanes ----
        int64_t slot = -1;
        const int tok = t0 + warp * 16 + lane;
        if (lane < 16 && tok < seq.x) slot = slot_of(p.page_table, b, tok, p.page_size, p.max_pages, p.num_pages, p.status);
        if (lane < 16) slots[warp * 16 + lane] = slot;
        const int row_bytes = Q8 ? p.d_c + 2 * p.d_r : 2 * (p.d_c + p.d_r);
        int hi = kNone, lo = kBad;                                      // largest and least exponent of the warp's tokens
        constexpr int kAhead = 4;                                       // tokens in flight
        const int per = p.d_c / 8;                                      // vectors of 8 latents a token
#pragma unroll 1
        for (int k0 = 0; k0 < 16; k0 += kAhead) {
            uint4 raw[kAhead][2];
            int64_t sl[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                sl[k] = __shfl_sync(0xffffffffu, slot, k0 + k);
                const uint8_t* src = p.kv + (sl[k] < 0 ? 0 : sl[k]) * (int64_t)row_bytes;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    raw[k][v] = make_uint4(0, 0, 0, 0);
                    const int c = lane + 32 * v;
                    if (sl[k] >= 0 && c < per) {
                        if constexpr (Q8) {
                            const uint2 u = *reinterpret_cast<const uint2*>(src + c * 8);
                            raw[k][v].x = u.x;
                            raw[k][v].y = u.y;
                        } else {
                            raw[k][v] = *reinterpret_cast<const uint4*>(src + c * 16);
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                float x[2][8];
                float top = 0.f;
                bool bad = false;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const uint32_t w[4] = {raw[k][v].x, raw[k][v].y, raw[k][v].z, raw[k][v].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (Q8) x[v][i] = e4m3_to_float((uint8_t)(w[i >> 2] >> (8 * (i & 3))));
                        else x[v][i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
                        top = fmaxf(top, fabsf(x[v][i]));
                        bad |= !isfinite(x[v][i]);
                    }
                }
                top = warp_max(top);
                bad = __any_sync(0xffffffffu, bad);
                int e = top > 0.f ? ilogbf(top) : kNone;                // of the latent, or of its codes
                int se = 0;
                if (Q8 && sl[k] >= 0) {
                    const float s = p.kv_scale[sl[k]];
                    bad |= !isfinite(s);
                    if (s == 0.f) e = kNone;
                    else se = ilogbf(s);
                    // a scale that is no power of two (none that this library writes): its mantissa goes into the codes
                    const float m = s == 0.f ? 0.f : ldexpf(s, -se);
                    if (m != 1.f) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i >> 3][i & 7] *= m;
                        if (e != kNone) e = ilogbf(top * fabsf(m));
                    }
                }
                const bool zero = bad || e == kNone;
                const int row = warp * 16 + k0 + k;
                const float f1 = zero ? 0.f : pow2i(-(e / 2)), f2 = zero ? 0.f : pow2i(-(e - e / 2));
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int c = lane + 32 * v;
                    if (c < per) {
                        uint32_t h[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            h[i] = zero ? 0u : pack_f16(x[v][2 * i] * f1 * f2, x[v][2 * i + 1] * f1 * f2);
                        *reinterpret_cast<uint4*>(sm + L.a + (c >> 3) * kBlock + sw128_offset(row, (c & 7) * 8)) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
                const int et = bad ? kBad : e == kNone ? kNone : e + se;
                if (lane == 0) exps[row] = et;
                if (et != kBad && et != kNone) { hi = max(hi, et); lo = min(lo, et); }
            }
        }
        if (lane == 0) { warp_hi[warp] = hi; warp_lo[warp] = lo; }
        fence_proxy_async_smem();
    }
    __syncthreads();
    int e_hi = kNone, e_lo = kBad;
#pragma unroll
    for (int i = 0; i < 8; ++i) { e_hi = max(e_hi, warp_hi[i]); e_lo = min(e_lo, warp_lo[i]); }
    // one exponent for the tile's values; bf16 where fp16 would not hold them beside one another
    const bool bf = e_hi != kNone && (e_hi - e_lo > 12 || e_hi > kMaxE || e_hi < -kMaxE);
    const int e_tile = e_hi == kNone ? 0 : min(max(e_hi, -kMaxE), kMaxE);
    if (part == 0 && tid == 0) p.tinfo[tile] = (e_tile + 64) | (bf ? 256 : 0);

    if (warp == 8) {
        // ---- weights ----
        const uint8_t* w = p.weights + kWeightTable + (size_t)n0 * kb * kBlock;
        const int all = (n1 - n0) * kb;
        int i = 0;
        for (; i < all; ++i) {
            const int s = i % kRing;
            if (i >= kRing && !dec::wait_bounded(&empty[s], ((i / kRing) - 1) & 1, p.status)) break;
            if (*(volatile int*)fail) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], kBlock);
                bulk_load(sm + L.ring + s * kBlock, w + (size_t)i * kBlock, kBlock, &full[s]);
            }
            __syncwarp();
        }
        if (lane == 0) {
            *(volatile int*)issued_s = i;
            if (i < all) *(volatile int*)fail = 1;
        }
    } else if (warp == 9) {
        // ---- products ----
        const uint32_t idesc = idesc_bf16(128, 128, 0, 0) & ~((1u << 7) | (1u << 10));      // fp16 operands
        int i = 0, n = n0;
        bool ok = true;
        for (; n < n1 && ok; ++n) {
            const int a = (n - n0) & 1;
            if (n - n0 >= 2) ok = dec::wait_bounded(&acc_empty[a], (((n - n0) >> 1) - 1) & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            for (int k = 0; k < kb; ++k, ++i) {
                const int s = i % kRing;
                if (!dec::wait_bounded(&full[s], (i / kRing) & 1, p.status)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t A = smem_u32(sm + L.a + k * kBlock), Bw = smem_u32(sm + L.ring + s * kBlock);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16(tmem + a * 128, smem_desc(A + kk * 32, 16, 1024, kSwizzle128B),
                                 smem_desc(Bw + kk * 32, 16, 1024, kSwizzle128B), idesc, (k > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(&empty[s]);
                    if (k == kb - 1) mma_commit(&acc_full[a]);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) *(volatile int*)fail = 1;
        if (elect_one()) mma_commit(done);
        __syncwarp();
    } else {
        // ---- results: thread = token, its warp's half of the 128 columns (one 64-column block) ----
        const int half = warp >> 2, row = 32 * (warp & 3) + lane;
        const int et = exps[row];
        const int64_t slot = slots[row];
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const int* we = reinterpret_cast<const int*>(p.weights);
        uint8_t* stage = sm + L.stage + half * kBlock;
        if (part == 0 && half == 0) {
            // RoPE keys: 16-byte pieces of 8 values, a 128-byte row by 8 (or 4) lanes
            const int row_bytes = Q8 ? p.d_c + 2 * p.d_r : 2 * (p.d_c + p.d_r);
            const int pieces = p.d_r / 8;
            for (int i = tid; i < kTile * pieces; i += 128) {
                const int r = i / pieces, c = i % pieces;
                const int64_t sl = slots[r];
                uint32_t h[4] = {0, 0, 0, 0};
                if (sl >= 0) {
                    const uint4 u = *reinterpret_cast<const uint4*>(p.kv + sl * (int64_t)row_bytes + (Q8 ? p.d_c : 2 * p.d_c) + c * 16);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = pack_f16(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
                }
                *reinterpret_cast<uint4*>(p.krope + (size_t)tile * kBlock + sw128_offset(r, c * 8)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        bool ok = true;                                                 // a thread that gave up still meets the barriers
        for (int n = n0; n < n1; ++n) {
            const int a = (n - n0) & 1;
            if (ok && (*(volatile int*)fail || !dec::wait_bounded(&acc_full[a], ((n - n0) >> 1) & 1, p.status))) {
                *(volatile int*)fail = 1;
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);                           // (the TMEM load is the warp's)
            if (!ok) {
                if (2 * n + half < blocks) {
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                }
                continue;
            }
            tc_fence_after();
            uint32_t v[64];
            tmem_ld64(tmem + lane_base + a * 128 + half * 64, v);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&acc_empty[a]);
            const int cb = 2 * n + half;
            if (cb < blocks) {
                const bool key = cb < p.G * nkb;
                float f;
                uint8_t* dst;
                bool as_bf = false;
                if (key) {
                    const int g = cb / nkb;
                    float al = 0.f;
                    if (slot >= 0) al = p.ak_f16 ? load_alpha<true>(p.ak, slot * p.G + g) : load_alpha<false>(p.ak, slot * p.G + g);
                    // NaN where the latent is not finite: rows that see the token become NaN, others do not
                    f = et == kBad ? __int_as_float(0x7fc00000) : et == kNone ? 0.f : ldexpf(al, et + we[g]);
                    dst = p.kc + ((size_t)tile * p.G * nkb + cb) * kBlock;
                } else {
                    f = et == kBad || et == kNone ? 0.f : ldexpf(1.f, et - e_tile);
                    as_bf = bf;
                    dst = p.v + ((size_t)tile * p.Gv * nvb + (cb - p.G * nkb)) * kBlock;
                }
                // the staging block is free once the last copy out of it has been read
                if ((warp & 3) == 0 && lane == 0) dec::bulk_wait_read_all();
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = __uint_as_float(v[8 * c + 2 * i]) * f, y = __uint_as_float(v[8 * c + 2 * i + 1]) * f;
                        h[i] = as_bf ? pack_bf16(x, y) : pack_f16(x, y);
                    }
                    *reinterpret_cast<uint4*>(stage + sw128_offset(row, c * 8)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async_smem();
                asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                if ((warp & 3) == 0 && lane == 0) {
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
                                 "r"(smem_u32(stage)), "r"(kBlock) : "memory");
                    dec::bulk_commit_group();
                }
            }
        }
        if ((warp & 3) == 0 && lane == 0) dec::bulk_wait_all();
    }
    __syncthreads();
    dec::wait_bounded(done, 0, p.status);
    if (*(volatile int*)fail && tid == 0) {
        const int issued = *(volatile int*)issued_s;
        for (int j = max(0, issued - kRing); j < issued; ++j) dec::wait_bounded(&full[j % kRing], (j / kRing) & 1, p.status);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <typename T>
int launch_query_type(const Params& p, cudaStream_t s) {
    const int64_t items = (int64_t)p.rows * p.H, per = kThreadsQ / 32 * kRowsWarp;
    const dim3 grid((unsigned)((items + per - 1) / per + 1)), block(kThreadsQ);
    cudaError_t e;
    if (p.d_h == 128) e = p.d_r == 64 ? launch_pdl(prefill_query_kernel<T, 128, 64>, grid, block, 0, s, p)
                                      : launch_pdl(prefill_query_kernel<T, 128, 32>, grid, block, 0, s, p);
    else e = p.d_r == 64 ? launch_pdl(prefill_query_kernel<T, 64, 64>, grid, block, 0, s, p)
                         : launch_pdl(prefill_query_kernel<T, 64, 32>, grid, block, 0, s, p);
    return e == cudaSuccess ? QKMLA_OK : QKMLA_ERR_CUDA;
}

}  // namespace

int launch_query(const Params& p, bool q_bf16, cudaStream_t s) {
    return q_bf16 ? launch_query_type<__nv_bfloat16>(p, s) : launch_query_type<float>(p, s);
}

int launch_expand(const Params& p, bool q8, cudaStream_t s) {
    const ExpandLayout L(p.d_c);
    auto k = q8 ? prefill_expand_kernel<true> : prefill_expand_kernel<false>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L.bytes) != cudaSuccess) return QKMLA_ERR_CUDA;
    // few tiles: their columns are cut over several CTAs
    const int nt = n_tiles(p.G, p.Gv, p.d_h, p.d_v);
    const int splits = max(1, min(nt, device_sm_count() / max(1, p.max_tiles)));
    if ((int64_t)p.max_tiles * splits > INT32_MAX) return QKMLA_ERR_UNSUPPORTED;
    return launch_pdl(k, dim3((unsigned)(p.max_tiles * splits)), dim3(kThreadsE), L.bytes, s, p, splits) == cudaSuccess ? QKMLA_OK
                                                                                                                      : QKMLA_ERR_CUDA;
}

}  // namespace pf
}  // namespace qkmla

using namespace qkmla;

static bool weights_served(int G, int Gv, int d_c, int d_h, int d_v) {
    return (d_h == 64 || d_h == 128) && (d_v == 64 || d_v == 128) && d_c % 64 == 0 && d_c <= 512 && G <= 512 && Gv <= 512;
}

extern "C" size_t qkmla_prefill_weights_size(int G, int G_v, int d_c, int d_h, int d_v) {
    if (G < 1 || G_v < 1 || d_c < 1 || d_h < 1 || d_v < 1 || !weights_served(G, G_v, d_c, d_h, d_v)) return 0;
    return pf::kWeightTable + (size_t)pf::n_tiles(G, G_v, d_h, d_v) * (d_c / 64) * pf::kBlock;
}

extern "C" int qkmla_prefill_pack_weights(const float* w_k, const void* w_v, int G, int G_v, int d_c, int d_h, int d_v,
                                          void* packed, void* stream) {
    if (G < 1 || G_v < 1 || d_c < 1 || d_h < 1 || d_v < 1 || !w_k || !w_v || !packed) return QKMLA_ERR_INVALID;
    if (((uintptr_t)w_k % 4) || ((uintptr_t)w_v % 2) || ((uintptr_t)packed % 16)) return QKMLA_ERR_INVALID;
    if (!weights_served(G, G_v, d_c, d_h, d_v)) return QKMLA_ERR_UNSUPPORTED;
    cudaStream_t s = (cudaStream_t)stream;
    return launch_pdl(pf::prefill_pack_kernel, dim3(G + G_v, d_c / 64), dim3(256), 0, s, w_k, (const __nv_bfloat16*)w_v, G, G_v, d_c,
                      d_h, d_v, (uint8_t*)packed) == cudaSuccess
               ? QKMLA_OK
               : QKMLA_ERR_CUDA;
}
