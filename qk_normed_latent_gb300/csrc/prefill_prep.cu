// qkmla_prefill, the kernels ahead of the attention, and the packing of its weights.
//
// prefill_pack_kernel   W^K (fp32) and W^V (bf16) as fp16 K-major blocks, each matrix times a power of two
//                       that brings its largest value into [1, 2): fp16's 11 bits hold W^V's 8 exactly and
//                       W^K to 2^-11, whatever the weights' scale.
// prefill_expand_kernel keys and values of the cached tokens, 128 a tile, on the tensor cores; its last block makes
//                       the plan of the attention's work (where the others fill every SM, as the first of them ends;
//                       given an SM of its own the calls took as long).
//
// Expansion.  A tile's latents are gathered once, as fp16 times 2^-e of each token, and stay in shared memory as A
// (M = 128 tokens, K = d_c) for all columns of W^K and W^V; weights stream through a ring, in N-tiles of 256 columns
// (128 up to d_c 256, where two CTAs fit on an SM).  The epilogue multiplies a token's key by alpha^k and its power of
// two, a value by the latter over the tile's largest.  Tiles that no row sees behind a window are left out (585 -> 555
// us of a windowed call), and a CTA takes an equal number of N-tiles, cutting a token tile where it must (223 -> 197
// us on a mixed batch).
//
// Bound: for large d_c the products (2 d_c (G d_h + G_v d_v) flops a token: 33.6 GFLOP, 17 us, for 16000 tokens at
// d_c 512 and 8 groups of 128 + 128), five fourths of that by shared memory's rate, and, per tile, the gather's latency and
// conversions in front of them (9 us a tile, of which the next tile's loads are prefetched).  Those 16000 tokens take
// 45-48 us, 29 % of tensor cycles; 131072 of the 8-bit cache 296 us.
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
        const int nb = blocks_per_tile(d_c);
        uint8_t* blk = blocks + ((size_t)(cb / nb) * (d_c / 64) + blockIdx.y) * (nb * (kBlock / 2));
        *reinterpret_cast<__half*>(blk + sw128_offset(cb % nb * 64 + j % 64, c)) = __float2half_rn(w);
    }
}

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------
constexpr int kThreadsE = 320;

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
    for (int i = 0; i < kThreadsE / 32; ++i) {
        if (i < warp) ahead += warps[i];
        sum += warps[i];
    }
    *all = sum;
    return ahead + s - v;
}

// `warps`: shared memory for a number a warp.
__device__ void make_plan(const Params& p, int64_t* warps) {
    const int tid = threadIdx.x;
    // sequences: lengths, first tiles, rows
    int64_t tiles = 0, tokens = 0, all;
    const int per = (p.B + kThreadsE - 1) / kThreadsE;
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b >= p.B) break;
        const int len = p.seq_lens[b];
        tiles += needed(p, len, p.chunk_start[b + 1] - p.chunk_start[b]).tiles;
        tokens += max(len, 0);
    }
    // chunk starts out of order: nothing is done, since ranges of query tiles could meet
    bool bad = false;
    for (int b = tid; b < p.B; b += kThreadsE) {
        const int r0 = p.chunk_start[b], r1 = p.chunk_start[b + 1];
        bad |= r0 < 0 || r0 > r1 || r1 > p.rows || (b == 0 && r0 != 0);
    }
    const bool ordered = !__syncthreads_or(bad);
    if (tid == 0 && !ordered) report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
    int64_t at = block_scan(tiles, warps, &all);
    int64_t sum;
    block_scan(tokens, warps, &sum);
    if (tid == 0 && sum > p.total_tokens) report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b >= p.B) break;
        int len = p.seq_lens[b];
        const int r0 = p.chunk_start[b], r1 = p.chunk_start[b + 1];
        const bool ok = len >= 0 && len <= (int64_t)p.max_pages * p.page_size;
        const Needed n = needed(p, len, r1 - r0);
        if (!ok) report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
        const bool fits = at + n.tiles <= p.max_tiles;     // no tile is read or written beyond the workspace
        p.seq[2 * b] = make_int4(ok && fits ? len : 0, (int)min(at, (int64_t)p.max_tiles), ordered ? r0 : 0, ordered ? r1 - r0 : 0);
        p.seq[2 * b + 1] = make_int4(n.gap, 0, 0, 0);
        at += n.tiles;
    }
    for (int j = tid; j < p.nq; j += kThreadsE) p.qinfo[2 * j] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    // query tiles: the tiles of tokens that any of their queries sees
    for (int b = tid >> 5; b < p.B; b += kThreadsE / 32) {
        const int4 s = p.seq[2 * b];
        const int n = s.w, j0 = first_slot(s.z, b, p.tq);
        for (int k = tid & 31; k * (int64_t)p.tq < n; k += 32) {
            const int i0 = k * p.tq, i1 = min(n, i0 + p.tq);
            const int lo = s.x - n + i0 + 1, hi = s.x - n + i1;        // causal lengths of the first and the last query
            const int total = hi > 0 ? (hi + kTile - 1) / kTile : 0;
            int head = total, gap = 0;
            if (const int64_t start = (int64_t)lo - p.window; p.window > 0 && start > 0) {
                const int from = (int)min(start / kTile, (int64_t)total);
                const int h = (int)((min((int64_t)p.sinks, start) + kTile - 1) / kTile);
                if (from > h) { head = h; gap = from - h; }
            }
            p.qinfo[2 * (j0 + k)] = make_int4(b, i0, total - gap, head);
            p.qinfo[2 * (j0 + k) + 1] = make_int4(gap, lo, i1 - i0, 0);
        }
    }
    __syncthreads();
    // the costs ahead of each place of the list
    const int places = p.ctas * p.deep, pq = (places + kThreadsE - 1) / kThreadsE;
    auto cost = [&](int m) {
        int u, j;
        if (!tile_of_place(p, m, u, j)) return 0;
        const int4 q = p.qinfo[2 * j];
        return q.x >= 0 ? q.z + kCostStart : 0;
    };
    int64_t mine_sum = 0;
    for (int k = 0; k < pq; ++k) {
        const int m = tid * pq + k;
        if (m >= places) break;
        mine_sum += cost(m);
    }
    int64_t ahead = block_scan(mine_sum, warps, &all);
    for (int k = 0; k < pq; ++k) {
        const int m = tid * pq + k;
        if (m >= places) break;
        p.pre[m] = ahead;
        ahead += cost(m);
    }
    if (tid == 0) p.pre[places] = all;
}

// ---------------------------------------------------------------------------
// keys and values
// ---------------------------------------------------------------------------
// C [128 tokens, d_c] x [W^K_0 .. W^K_{G-1} | W^V_0 ..] in N-tiles of 256 columns (128 up
// to d_c = 256, where two CTAs share an SM and its TMEM).  The latents lie in shared
// memory while their tile is worked on (d_c / 64 blocks), each token times a power of two of its own that brings its
// largest value into [1, 2): exact as fp16 for a bf16 or an 8-bit latent, but for what lies 2^-14 below that
// value.  Warps 0-7 gather and convert them, then take the results out of TMEM: a key row is scaled by the
// stored alpha^k, a value row by its share of the tile's common exponent.  A thread holds 64 columns of a token,
// one 128-byte line of a block; quads of lanes exchange pieces so that each store writes whole lines.  Warp 8 streams the packed weights through a
// ring, warp 9 issues the products (M = 128, N = 128 or 256, K = 64 a stage), the accumulator double-buffered.
//
// Bound: shared memory.  A stage's four products take 512 cycles of the tensor core, but read 4 x (4 KB of latents + 8 KB of
// weights) while 32 KB of the next weights are written: 80 KB, 640 cycles at 128 bytes, and 640 a stage is what it takes.
// (Two CTAs that bring half of each stage for both were no faster: L2 does not hold it back.)  The ring takes all the shared
// memory that the latents leave (three stages at d_c = 512).  Few tiles: their columns are cut over several CTAs.
constexpr int kRingMax = 3;

// blocks of the latents, a ring of three stages of 32 KB or two of 16 KB
__host__ __device__ inline int expand_bytes(int d_c) { return (d_c / 64 + (d_c <= 256 ? 2 : 2 * kRingMax)) * kBlock + 1024 + 2048; }

struct __align__(16) ExpandShared {
    uint64_t full[kRingMax], empty[kRingMax];
    uint64_t acc_full[2], acc_empty[2], a_full, done;
    int exps[2][kTile];
    int hi[2][8], lo[2][8];
    uint32_t tmem;
    int fail, issued;
};
static_assert(sizeof(ExpandShared) <= 2048, "beside the blocks");

// The sequence of a tile of the workspace, by the tiles of those ahead of it; tiles are asked for in rising order, so the
// next tile's is mostly the same one.  Whole warp.
struct Sequence {
    int b = 0, first = 0, last = 0, len = 0, head = 0, gap = 0;         // its tiles: [first, last)
    int from = 0;                                          // where its first row's window starts
    int b0 = 0, ahead = 0;                                 // where the next search starts: sequences, and tiles ahead of them
    __device__ __forceinline__ bool find(const Params& p, int tile) {
        if (tile < last) return tile >= first;
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (; b0 < p.B; b0 += 32) {
            const int at = b0 + lane;
            const int n = at < p.B ? p.seq_lens[at] : 0;
            const int rows = at < p.B ? p.chunk_start[at + 1] - p.chunk_start[at] : 0;
            const Needed d = needed(p, n, rows);
            int s = d.tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            const int all = __shfl_sync(0xffffffffu, s, 31);
            if (ahead + all > tile) {
                const int l = __ffs(__ballot_sync(0xffffffffu, ahead + s > tile)) - 1;
                b = b0 + l;
                len = __shfl_sync(0xffffffffu, n, l);
                head = __shfl_sync(0xffffffffu, d.head, l);
                gap = __shfl_sync(0xffffffffu, d.gap, l);
                from = p.window > 0 ? (int)max((int64_t)len - __shfl_sync(0xffffffffu, rows, l) + 1 - p.window, (int64_t)0) : 0;
                last = ahead + __shfl_sync(0xffffffffu, s, l);
                first = last - __shfl_sync(0xffffffffu, d.tiles, l);
                return true;
            }
            ahead += all;
        }
        last = first = 1 << 30;                            // behind the last sequence
        return false;
    }
    // Whether some row sees token t.  What none sees is taken as zeros, here and in all that is formed from a tile's tokens
    // together, and its page is not looked up.
    __device__ __forceinline__ bool sees(const Params& p, int t) const { return t < len && (t >= from || t < p.sinks); }
    // The first token of a tile.
    __device__ __forceinline__ int token(int tile) const { return (tile - first < head ? tile - first : tile - first + gap) * kTile; }
};

// A CTA's share of the work, in N-tiles of all tiles: where the tiles are fewer than CTAs, each CTA a part of one tile;
// else equal shares, whose ends may cut a tile (its latents are then gathered twice).  Whole warp.
struct Share {
    int64_t at, end;
    __device__ __forceinline__ Share(const Params& p, int nt, int cta, int ctas) {
        const int lane = threadIdx.x & 31;
        int64_t tiles = 0;
        for (int b = lane; b < p.B; b += 32) tiles += needed(p, p.seq_lens[b], p.chunk_start[b + 1] - p.chunk_start[b]).tiles;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        tiles = min(tiles, (int64_t)p.max_tiles);
        at = end = 0;
        if (tiles == 0) return;
        if (tiles <= ctas) {
            const int parts = min(nt, (int)(ctas / tiles)), tile = cta / parts, part = cta - tile * parts;
            if (tile >= tiles) return;
            at = (int64_t)tile * nt + nt * part / parts;
            end = (int64_t)tile * nt + nt * (part + 1) / parts;
        } else {
            // (with few N-tiles a tile is cheaper done whole than gathered twice: 36 against 44 us for 480 tiles of four)
            const int cut = nt >= 8 ? 1 : nt;
            at = tiles * nt / cut * cta / ctas * cut;
            end = tiles * nt / cut * (cta + 1) / ctas * cut;
        }
    }
    // The next tile and its N-tiles [n0, n1).
    __device__ __forceinline__ bool next(int nt, int& tile, int& n0, int& n1) {
        if (at >= end) return false;
        tile = (int)(at / nt);
        n0 = (int)(at - (int64_t)tile * nt);
        n1 = (int)min((int64_t)nt, n0 + (end - at));
        at += n1 - n0;
        return true;
    }
};

// A token's latents, NV vectors of 8 a lane, to row r of the tile's blocks as fp16 times 2^-e, e the exponent of its largest
// value.  Returns the token's exponent (with its scale's), kNone for zeros, kBad (and zeros) where one is not finite.
template <bool Q8, int NV>
__device__ __forceinline__ int convert_token(const uint4 (&raw)[NV], float scale, int per, uint8_t* blocks, int r, int lane) {
    uint32_t h[NV][4];
    int e;
    bool bad;
    if constexpr (Q8) {
        // codes are fp16 values: two at a time throughout, the largest magnitude by their patterns (NaN above all numbers)
        __half2 x[NV][4];
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t w[2] = {raw[v].x, raw[v].y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[v][i] = __half2(__half2_raw(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3)));
                top = __vmaxu2(top, *reinterpret_cast<const uint32_t*>(&x[v][i]) & 0x7fff7fffu);
            }
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        const uint32_t sb = __float_as_uint(scale);
        bad = most > 0x7c00u || (sb & 0x7f800000u) == 0x7f800000u;
        e = most == 0 || scale == 0.f ? kNone : (int)(most >> 10) - 15;      // (the least code, 2^-9, is a normal fp16 number)
        __half f = __ushort_as_half((unsigned short)((15 - (e == kNone ? 0 : e)) << 10));
        if ((sb & 0x807fffffu) == 0 || bad || e == kNone) {                  // a power of two, as this library writes them
            e = e == kNone ? kNone : e + (int)(sb >> 23) - 127;
            const __half2 f2 = __half2half2(f);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[v][i] = __hmul2(x[v][i], f2);
        } else {                                                             // any other scale leaves its mantissa in the codes
            const int se = ilogbf(scale);
            const float m = ldexpf(scale, -se), t = __half2float(__ushort_as_half((unsigned short)most)) * fabsf(m);
            e = ilogbf(t);
            const float g = m * pow2i(-e);
            e += se;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[v][i] = __floats2half2_rn(__low2float(x[v][i]) * g, __high2float(x[v][i]) * g);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) h[v][i] = *reinterpret_cast<const uint32_t*>(&x[v][i]);
    } else {
        // the largest magnitude by the bf16 patterns, two at a time
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t w[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
        bad = most >= 0x7f80u;
        e = most == 0 ? kNone : min(max((int)(most >> 7) - 127, -126), 126);
        const float f = e == kNone || bad ? 0.f : pow2i(-e);
        const uint64_t f2 = dec::f2(f, f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t w[4] = {raw[v].x, raw[v].y, raw[v].z, raw[v].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 y = dec::f2_unpack(dec::f2_mul(dec::f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), f2));
                h[v][i] = pack_f16(y.x, y.y);
            }
        }
    }
    const bool zero = bad || e == kNone;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = lane + 32 * v;
        if (c < per)
            *reinterpret_cast<uint4*>(blocks + (c >> 3) * kBlock + sw128_offset(r, (c & 7) * 8)) =
                zero ? make_uint4(0, 0, 0, 0) : make_uint4(h[v][0], h[v][1], h[v][2], h[v][3]);
    }
    return bad ? kBad : e;
}

// NV: vectors of 8 latents a lane, d_c up to 256 NV; at 1 two CTAs fit on an SM, one gathering while the other multiplies.
template <bool Q8, int NV>
__global__ void __launch_bounds__(kThreadsE, NV == 1 ? 2 : 1) prefill_expand_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    constexpr int kRing = NV == 1 ? 2 : kRingMax;
    constexpr int NB = NV == 1 ? 2 : 4;                     // column blocks of an N-tile
    constexpr int kStage = NB * (kBlock / 2);
    constexpr uint32_t kCols = NB * 64;
    const int kb = p.d_c / 64;
    uint8_t* ring = sm + kb * kBlock;
    ExpandShared* sh = reinterpret_cast<ExpandShared*>(ring + kRing * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nkb = p.d_h / 64, nvb = p.d_v / 64;
    const int blocks = column_blocks(p.G, p.Gv, p.d_h, p.d_v), nt = (blocks + NB - 1) / NB;
    const int ctas = gridDim.x - 1;

    if (blockIdx.x == ctas) {
        pdl_wait();                                        // the workspace may still be in use
        pdl_trigger();
        make_plan(p, reinterpret_cast<int64_t*>(sm));
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) { mbar_init(&sh->full[i], 1); mbar_init(&sh->empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&sh->acc_full[i], 1); mbar_init(&sh->acc_empty[i], 8); }
        mbar_init(&sh->a_full, 8);
        mbar_init(&sh->done, 1);
        sh->fail = 0;
        sh->issued = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&sh->tmem, 2 * kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    int* fail = &sh->fail;
    pdl_wait();
    pdl_trigger();

    if (warp == 8) {
        // ---- weights ----
        Share share(p, nt, blockIdx.x, ctas);
        int i = 0, tile, n0, n1;
        bool ok = true;
#pragma unroll 1
        while (ok && share.next(nt, tile, n0, n1)) {
            const uint8_t* w = p.weights + kWeightTable + (size_t)n0 * kb * kStage;
            if (lane == 0) {
#pragma unroll 1
                for (int q = 0; q < (n1 - n0) * kb; ++q, ++i) {
                    const int s = i % kRing;
                    if (i >= kRing && !(ok = wait_or_fail(&sh->empty[s], ((i / kRing) - 1) & 1, fail))) break;
                    mbar_arrive_expect_tx(&sh->full[s], kStage);
                    bulk_load(ring + s * kStage, w + (size_t)q * kStage, kStage, &sh->full[s]);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) *(volatile int*)&sh->issued = i;
    } else if (warp == 9) {
        // ---- products: each barrier is looked at while the ones ahead of its use are being taken ----
        constexpr uint32_t idesc = idesc_bf16(128, kCols, 0, 0) & ~((1u << 7) | (1u << 10));      // fp16 operands
        const uint32_t a_desc = desc_low(sm, 16), w_desc = desc_low(ring, 16);
        Share share(p, nt, blockIdx.x, ctas);
        int i = 0, n = 0, it = 0, tile, n0, n1;            // blocks, N-tiles and tiles so far
        bool ok = true;
#pragma unroll 1
        while (ok && share.next(nt, tile, n0, n1)) {
            if (elect_one()) {
                ok = wait_or_fail(&sh->a_full, it & 1, fail);
                bool seen = false;
                const int blocks_all = (n1 - n0) * kb;
                int k = 0;
#pragma unroll 1
                for (int q = 0; q < blocks_all && ok; ++q, ++i) {
                    const int s = i % kRing, a = n & 1;
                    if (k == 0 && n >= 2 && !(ok = wait_or_fail(&sh->acc_empty[a], ((n >> 1) - 1) & 1, fail))) break;
                    if (!seen && !(ok = wait_or_fail(&sh->full[s], (i / kRing) & 1, fail))) break;
                    if (k == 0) tc_fence_after();
                    const uint32_t A = a_desc + k * (kBlock >> 4), W = w_desc + s * (kStage >> 4), d = tmem + a * kCols;
                    mma_ss(d, A, W, idesc, k > 0 ? 1u : 0u);
                    mma_ss(d, A + 2, W + 2, idesc, 1u);
                    const int s2 = (i + 1) % kRing;
                    seen = mbar_test_wait(&sh->full[s2], ((i + 1) / kRing) & 1);
                    mma_ss(d, A + 4, W + 4, idesc, 1u);
                    mma_ss(d, A + 6, W + 6, idesc, 1u);
                    mma_commit(&sh->empty[s]);
                    if (++k == kb) {
                        mma_commit(&sh->acc_full[a]);
                        k = 0;
                        ++n;
                    }
                }
            }
            __syncwarp();
            // (the counts are the elected lane's; the others' follow from the item's size)
            ok = __all_sync(0xffffffffu, ok);
            ++it;
            i = __reduce_max_sync(0xffffffffu, i);
            n = __reduce_max_sync(0xffffffffu, n);
        }
        if (elect_one()) mma_commit(&sh->done);
        __syncwarp();
    } else {
        const int row_bytes = Q8 ? p.d_c + 2 * p.d_r : 2 * (p.d_c + p.d_r);
        const int per = p.d_c / 8;                          // vectors of 8 latents a token
        const int* we = reinterpret_cast<const int*>(p.weights);
        Share share(p, nt, blockIdx.x, ctas);
        Sequence seq;
        int n = 0, it = 0, tile, n0, n1;
        bool ok = true;
#pragma unroll 1
        while (ok && share.next(nt, tile, n0, n1)) {
            seq.find(p, tile);
            const int t0 = seq.token(tile), buf = it & 1;
            // ---- gather: a warp's 16 tokens, their slots by its first 16 lanes ----
            const int row = 32 * (warp & 3) + lane;          // this thread's token in the results
            const int mine = t0 + (lane < 16 ? warp * 16 + lane : row);
            auto slot_at = [&](int t) {
                return seq.sees(p, t) ? slot_of(p.page_table, seq.b, t, p.page_size, p.max_pages, p.num_pages, p.status) : (int64_t)-1;
            };
            const int64_t slot = slot_at(mine);              // (of lanes from 16 on it is not used)
            const int64_t row_slot = slot_at(t0 + row);
            float scale = 0.f;                               // of lane's token, 8-bit cache
            if (Q8 && lane < 16 && slot >= 0) scale = p.kv_scale[slot];
            int hi = kNone, lo = kBad;                       // largest and least exponent of the warp's tokens
            constexpr int kAhead = 8;                        // tokens in flight
#pragma unroll 1
            for (int k0 = 0; k0 < 16; k0 += kAhead) {
                uint4 raw[kAhead][NV];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int64_t sl = __shfl_sync(0xffffffffu, slot, k0 + k);
                    const uint8_t* src = p.kv + (sl < 0 ? 0 : sl) * (int64_t)row_bytes;
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        raw[k][v] = make_uint4(0, 0, 0, 0);
                        const int c = lane + 32 * v;
                        if (sl >= 0 && c < per) {
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
                    const int r = warp * 16 + k0 + k;
                    const float s = __shfl_sync(0xffffffffu, scale, k0 + k);
                    const int e = convert_token<Q8, NV>(raw[k], s, per, sm, r, lane);
                    if (lane == 0) sh->exps[buf][r] = e;
                    if (e != kBad && e != kNone) { hi = max(hi, e); lo = min(lo, e); }
                }
            }
            if (n0 == 0) {
                // RoPE keys of the warp's tokens: 16-byte pieces of 8 values, a row by 8 (or 4) lanes, all in flight at once
                const int pieces = p.d_r / 8;
                uint4 u[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = lane + 32 * q, k = i / pieces, c = i - k * pieces;
                    const int64_t sl = __shfl_sync(0xffffffffu, slot, k & 15);
                    u[q] = make_uint4(0, 0, 0, 0);
                    if (k < 16 && sl >= 0) u[q] = *reinterpret_cast<const uint4*>(p.kv + sl * (int64_t)row_bytes + (Q8 ? p.d_c : 2 * p.d_c) + c * 16);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = lane + 32 * q, k = i / pieces, c = i - k * pieces;
                    if (k >= 16) continue;
                    const uint32_t w[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = pack_f16(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
                    *reinterpret_cast<uint4*>(p.krope + (size_t)tile * kBlock + sw128_offset(warp * 16 + k, c * 8)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
            if (lane == 0) { sh->hi[buf][warp] = hi; sh->lo[buf][warp] = lo; }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->a_full);
            // the next tile's rows into L2, where it is of the same sequence
            if (share.at < share.end && tile + 1 < seq.last && lane < 16) {
                const int64_t sl = slot_at(seq.token(tile + 1) + warp * 16 + lane);
                if (sl >= 0)
                    for (int i = 0; i < row_bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.kv + sl * (int64_t)row_bytes + i));
            }
            const int half = warp >> 2;
            auto alpha_of = [&](int cb) {                    // of the key block's group
                if (cb >= p.G * nkb || row_slot < 0) return 0.f;
                const int64_t i = row_slot * p.G + cb / nkb;
                return p.ak_f16 ? load_alpha<true>(p.ak, i) : load_alpha<false>(p.ak, i);
            };
            float al = alpha_of(NB * n0 + half * (NB / 2));
            ok = wait_or_fail(&sh->a_full, it & 1, fail);
            ++it;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            int e_hi = kNone, e_lo = kBad;
#pragma unroll
            for (int i = 0; i < 8; ++i) { e_hi = max(e_hi, sh->hi[buf][i]); e_lo = min(e_lo, sh->lo[buf][i]); }
            const TileScale ts(e_hi, e_lo);
            const bool bf = ts.bf;
            const int e_tile = ts.e;
            if (n0 == 0 && tid == 0) p.tinfo[tile] = ts.packed();
            // ---- results: thread = token, its warp's half of the 128 columns (one 64-column block) ----
            const int et = sh->exps[buf][row];
            const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
#pragma unroll 1
            for (int q = n0; q < n1; ++q, ++n) {
                const int a = n & 1;
                ok = wait_or_fail(&sh->acc_full[a], (n >> 1) & 1, fail);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int sub = 0; sub < NB / 2; ++sub) {
                const int cb = NB * q + half * (NB / 2) + sub;
                const float al_now = al;
                al = alpha_of(sub + 1 < NB / 2 ? cb + 1 : cb + 1 + NB / 2);
                uint32_t v[64];
                tmem_ld64(tmem + lane_base + a * kCols + (half * (NB / 2) + sub) * 64, v);
                tmem_wait_ld();
                if (sub == NB / 2 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->acc_empty[a]);
                }
                if (cb >= blocks) continue;
                const bool key = cb < p.G * nkb;
                float f;
                uint8_t* dst;                                // of the block
                int split = 0;                               // what rows from 64 on add (a matrix's values lie by 64 tokens, then by 64 columns)
                if (key) {
                    // NaN where the latent is not finite: rows that see the token become NaN, others do not
                    f = et == kBad ? __int_as_float(0x7fc00000) : et == kNone ? 0.f : ldexpf(al_now, et + we[cb / nkb]);
                    dst = p.kc + ((size_t)tile * p.G * nkb + cb) * kBlock;
                } else {
                    f = et == kBad || et == kNone ? 0.f : ldexpf(1.f, et - e_tile);
                    const int m = (cb - p.G * nkb) / nvb, c = (cb - p.G * nkb) % nvb;
                    dst = p.v + ((size_t)tile * p.Gv + m) * nvb * kBlock + c * (kBlock / 2);
                    split = (nvb - 1) * (kBlock / 2);
                }
                const bool as_bf = bf && !key;
                const uint64_t f2 = dec::f2(f, f);
                uint32_t h[4][8];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 x = dec::f2_unpack(dec::f2_mul(dec::f2(__uint_as_float(v[16 * c + 2 * i]), __uint_as_float(v[16 * c + 2 * i + 1])), f2));
                        h[c][i] = as_bf ? pack_bf16(x.x, x.y) : pack_f16(x.x, x.y);
                    }
                quad_transpose(h, lane);
                const int r0 = row & ~3;
                dst += r0 * 128 + (r0 >= 64 ? split : 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {                // row r0 + k: two neighbouring 16-byte pieces, in swizzled order
                    const int r = r0 + k;
                    uint8_t* to = dst + k * 128 + (((lane & 3) ^ ((r >> 1) & 3)) << 5);
                    const uint32_t (&one)[8] = h[k];
                    if (k & 1) st_global_v8(to, {one[4], one[5], one[6], one[7]}, {one[0], one[1], one[2], one[3]});
                    else st_global_v8(to, {one[0], one[1], one[2], one[3]}, {one[4], one[5], one[6], one[7]});
                }
                }
            }
        }
    }
    __syncthreads();
    wait_or_fail(&sh->done, 0, fail);
    if (*(volatile int*)fail && tid == 0) {
        report(p.status, QKMLA_ERR_TIMEOUT);
        const int issued = *(volatile int*)&sh->issued;
        for (int j = max(0, issued - kRing); j < issued; ++j) dec::wait_bounded(&sh->full[j % kRing], (j / kRing) & 1, p.status);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kCols);
    }
}

template <bool Q8, int NV>
int launch_expand_as(const Params& p, cudaStream_t s) {
    auto k = prefill_expand_kernel<Q8, NV>;
    const int bytes = expand_bytes(p.d_c), sms = device_sm_count() * (NV == 1 ? 2 : 1);
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return QKMLA_ERR_CUDA;
    const int64_t most = (int64_t)p.max_tiles * n_tiles(p.G, p.Gv, p.d_h, p.d_v, p.d_c);
    const int ctas = (int)min((int64_t)sms, most);
    return launch_pdl(k, dim3((unsigned)(ctas + 1)), dim3(kThreadsE), bytes, s, p) == cudaSuccess ? QKMLA_OK : QKMLA_ERR_CUDA;
}

}  // namespace

int launch_expand(const Params& p, bool q8, cudaStream_t s) {
    if (p.d_c <= 256) return q8 ? launch_expand_as<true, 1>(p, s) : launch_expand_as<false, 1>(p, s);
    return q8 ? launch_expand_as<true, 2>(p, s) : launch_expand_as<false, 2>(p, s);
}

}  // namespace pf
}  // namespace qkmla

using namespace qkmla;

static bool weights_served(int G, int Gv, int d_c, int d_h, int d_v) {
    return (d_h == 64 || d_h == 128) && (d_v == 64 || d_v == 128) && d_c % 64 == 0 && d_c <= 512 && G <= 512 && Gv <= 512;
}

extern "C" size_t qkmla_prefill_weights_size(int G, int G_v, int d_c, int d_h, int d_v) {
    if (G < 1 || G_v < 1 || d_c < 1 || d_h < 1 || d_v < 1 || !weights_served(G, G_v, d_c, d_h, d_v)) return 0;
    return pf::kWeightTable + (size_t)pf::n_tiles(G, G_v, d_h, d_v, d_c) * (d_c / 64) * pf::blocks_per_tile(d_c) * (pf::kBlock / 2);
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
