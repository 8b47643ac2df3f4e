// Tensor-core decode kernel for the 8-bit latent cache (tcgen05 + TMEM + TMA).
//
// Definition (qkmla.h): with c^_t = s_t x_t, x_t the e4m3 codes and s_t the token's
// power-of-two scale,
//     l_{i,t,h} = scale (alpha^q_{i,h} alpha^k_{t,g(h)} s_t (q~_{i,h} . x_t) + q^r_{i,h} . k^r_t)
//     o_{i,h}   = sum_t p_t s_t x_t,  p = softmax over the tokens query i sees.
//
// The codes go to the tensor core as they are stored (kind::f8f6f4: no conversion
// pass, half the shared memory of bf16), and the other operand of each product is
// split into two 8-bit parts, a = hi + lo, hi = e4m3(a), lo = a - hi rounded.  For the
// bf16 query (lo in e4m3) the sum is exact down to 2^-18 of the row's largest value (8
// significant bits in two times 4); a weight (lo in e5m2, or in e4m3 with an accumulator
// and a unit of its own) is off by at most 2^-8, like a bf16 rounding, or, where it is
// small, by a step of lo whose sign depends on the token's place alone (see below).  The
// RoPE query is two bf16 parts (2^-16).  A tcgen05.mma with
// K = 32 costs 45 cycles up to N = 32, 48 at N = 64 and 65 at N = 128 (M = 64 or 128,
// K-major or MN-major, measured), so both parts as rows of one operand cost little more
// than one.
//
// Orientation.  A CTA owns up to 64 query rows (heads x query tokens) and a range of
// 64-token tiles; tokens are the M of the logit product, latents that of the output:
//   S   = X_tile [Q_hi | Q_lo]^T    M = 64 tokens, N = 2 ROWS, K = d_c              (e4m3)
//   R   = Kr_tile [Qr_hi | Qr_lo]^T M = 64 tokens, N = 2 ROWS, K = d_r              (bf16)
//   O^T += X_tile^T [P_hi | P_lo]   M = 128 latents of a chunk, K = 64 tokens       (e4m3)
// With 64 rows and 512 latents S, R and O^T fill TMEM's 512 columns (one S buffer; P_hi
// and P_lo then go into one accumulator by two MMAs), and the query parts, 80 KB, leave
// room for three 43 KB stages.  64 rows a CTA rather than 32 with 128-token tiles halve
// what a row costs in shared-memory traffic and loads (4400 cycles for 32 rows x 128 tokens
// against 2340 for 64 x 64).  A softmax thread is a token and 8 rows: the token's scale,
// alpha^k and mask are its registers, the row sums stay in registers until the end, and the
// running maximum is only looked at (one vote a tile) -- it moves when a weight outgrows e4m3.
//
// Weights in units of the output.  P carries s_t, so that the output product runs on
// the bare codes: p_{t,h} = 16 2^(x_t - m_h) s_t 2^(m_h - v_h) with m_h the running
// maximum of the logits x (log2) and v_h that of x + log2 s, the largest single
// contribution -- a maximum over logits alone would push the weights of ordinary
// tokens beside an outlier's scale below e4m3's range.  m and v are integers: every
// rescale is a power of two, hence exact.  A move costs a tile's time (2350 cycles: O^T is
// rescaled, so the previous output product has to end first), and the slowest CTA of a call
// had 20 when the first tile's largest contribution was put at 8 of at most 256 (64 x 4096
// tokens 111 us against 95, 4 x 262144 301 against 279).  It sits at 2 .. 4 of at most 448 and a
// move is rare.
//
// Small weights.  The denominator counts a weight in full, so what its 8-bit parts lose must
// not add up over the tokens: one token may outweigh each of 2^18 others that outweigh it
// together (rounded to nearest, 2^-18 of the largest each, they vanished and half of the
// result with them).  Two things keep the sum right.  (1) Below 2^-6, where hi has fewer than
// its 4 bits, lo is rounded up or down in proportion: a dither of one step goes in before it
// is cut, a token's place in a Weyl sequence (golden ratio), even over any run of tokens and
// the same on every call.  What N tokens are off by is then sqrt(N) steps of at most 2^-13,
// not N of them.  (2) Long items raise their units, by one move, when some tiles have shown
// what is large: more than 32 tiles after 4 of them, to 4 .. 8 for the largest contribution in
// the first and the fifth tile (8 .. 16 in more than 128 tiles, and from 16 tiles on where lo has
// its own accumulator), more than 256 after 128 again, to 64 .. 128.  Few later ones exceed that.
// A step is then at most 2^-14 (2^-15, 2^-16, 2^-19) of the largest for 2^11 (2^13, 2^14, more)
// tokens.  Against 64 bits, one token over a flat background of 2000 (8000, 16000, 262144), with
// latents of up to 3 times its norm: 3.7e-3 (3.6e-3, 3.4e-3, 2.8e-3) of the result's norm at the
// worst ratio.  Cost: 64 x 4096 tokens 89 -> 92 us, 4 x 262144 269 -> 276, windowed 99 -> 96,
// few rows nothing.
//
// What bounds it (512 / 64, 64 rows): a tile takes about 2380 cycles.  Its MMAs alone, one after
// the other, would take 2076 (20 x 65 + 16 x 48; the pipe's own counter says 1880 busy) and shared
// memory at 128 bytes a cycle about 2200: the 36 MMAs read 6 KB of operands each, 216 KB, the tile
// is 43 KB, P and the softmax's loads ~20 KB.  (With the query parts as the M = 128 operand an MMA
// takes 48 cycles and S fits twice, but it reads the same 6 KB and the softmax, a thread to a row,
// loads twice as much: 2900 cycles.)  64 sequences x 4096 tokens x 128 heads: 92 us (2.13 TB/s,
// 0.79 PFLOP/s counted once; the two parts make it 1.6) on 128 of the 152 SMs, of which ~13 us are
// the start and end of the items; 4 x 262144 tokens: 279 us (1.05 PFLOP/s).  The bf16 pair kernel
// takes 119 and 342 us.  With 16 rows (d_c = 256) the calls are latency-bound: 16 sequences of
// 1k-8k tokens 14 us.
//
// Warps: 0 TMA producer (+ TMEM owner), 1 logit MMAs, 2 output MMAs (each issue loop in
// one elected lane: a branch on the lane number costs ~88 cycles an MMA), then softmax and
// epilogue in groups of 4 warps, 16 rows a group.  All waits are bounded (2 s).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "decode_common.cuh"
#include "decode_sched.cuh"
#include "tc_ptx.cuh"

namespace qkmla {
namespace {

using namespace tc;
using namespace dec;

constexpr int kT = 64;               // tokens per tile
constexpr int kHpt = 8;              // query rows of a softmax thread
constexpr uint32_t kTmemCols = 512;
constexpr float kPUnit = 16.f;       // P of a contribution of 2^v
constexpr float kTopP = 448.f;       // a P above this (e4m3's largest value) moves the running maxima,
constexpr float kTopE = 1.09951163e12f;   // and so does 2^(x - m) above 2^40, fp32's margin for the row sums
constexpr float kLoUnit = 16.f;      // of the remainder's column where it has an accumulator of its own
constexpr int kSettle1 = 4, kSettle2 = 128;            // tiles after which items of more than
constexpr int kSettleFrom1 = 32, kSettleFrom2 = 256;   // this many raise their units (two accumulators: 16, at no cost)
constexpr int kSettleMore = 128;                       // tiles from which the first time is one binade more (always)

template <int DC, int DR, int ROWS>
struct Q8Layout {
    static constexpr int kN = 2 * ROWS;                       // hi and lo rows
    static constexpr int kGroups = ROWS / 16;                 // softmax groups of 4 warps
    static constexpr int kThreads = 96 + 128 * kGroups;
    static constexpr int kBlocks = DC / 128;                  // 128-column blocks = output chunks
    static constexpr int kRopeRow = DR * 2;                   // bytes: 128 (SW128) or 64 (SW64)
    static constexpr int kQLat = kBlocks * kN * 128;
    static constexpr int kQRope = kN * kRopeRow;
    static constexpr int kQ = (kQLat + kQRope + 1023) / 1024 * 1024;
    // TMEM: one or two buffers of S_hi S_lo R_hi R_lo, then O^T with P_hi and P_lo as columns of one operand
    // (two accumulators, added in the epilogue) or, where that does not fit, in two passes over one
    static constexpr bool kStacked = 4 * ROWS + kBlocks * kN <= 512;
    static constexpr int kON = kStacked ? kN : ROWS;          // columns of a chunk's accumulator
    static constexpr int kNsb = 8 * ROWS + kBlocks * kON <= 512 ? 2 : 1;
    static constexpr uint32_t kColO = kNsb * 4 * ROWS;
    // A stage holds a tile in groups of 8 tokens: kBlocks (with d_r = 64 one more, the RoPE key) blocks of
    // 8 tokens x 128 bytes, the swizzle's atom, as one TMA box of a page piece leaves them.  P (kN
    // bytes a token) takes the RoPE key's place where it fits.
    static constexpr bool kRopeIn = DR == 64;
    static constexpr bool kPOwn = kN > kRopeRow;
    static constexpr int kGroup = (kBlocks + (kRopeIn ? 1 : 0)) * 1024;
    static constexpr int kOffRope = kRopeIn ? kBlocks * 1024 : kT / 8 * kGroup;
    static constexpr int kRopeGroup = kRopeIn ? kGroup : 8 * kRopeRow;
    static constexpr int kOffOwn = kT / 8 * kGroup + (kRopeIn ? 0 : kT * kRopeRow);
    static constexpr int kOffP = kPOwn ? kOffOwn : kOffRope;
    static constexpr int kPGroup = kPOwn ? 8 * kN : kRopeGroup;
    static constexpr int kOffAk = kOffOwn + (kPOwn ? kT * kN : 0);
    static constexpr int kOffScale = kOffAk + kT * kMaxG * 4;
    static constexpr int kStage = (kOffScale + kT * 4 + 1023) / 1024 * 1024;
    // per-row floats: coef, m, v, t, f, corr, inv, and the column maxima of 4 warps (two kinds)
    static constexpr int kRowFloats = 7 * ROWS + 8 * ROWS;
    static constexpr int kMisc = 512 + kRowFloats * 4 + 1024;
    static constexpr int kStatic = (int)sizeof(SchedSmem) + 256;
    static constexpr int kNst = std::min(6, (232448 - kQ - kMisc - kStatic) / kStage);
    static constexpr int kOffStage = kQ;
    static constexpr int kOffMisc = kQ + kNst * kStage;
    static constexpr int kNumBars = 4 * kNst + 2 * kNsb + 2;
    static constexpr int kBytes = kOffMisc + kMisc;
    static_assert(kNst >= 3 && kOffAk % 1024 == 0 && kOffOwn % 1024 == 0, "three stages, aligned atoms");
    static_assert(kColO + kBlocks * kON <= kTmemCols, "TMEM budget");
    static_assert(kNumBars * 8 + 16 <= 512 && kBytes + kStatic <= 232448, "shared memory budget");
};

struct Q8Params {
    const __nv_bfloat16* qt;
    const float *aq, *qr, *grq;
    const uint8_t* ak;           // fp32 or fp16
    const float* kv_scale;
    const int32_t *seq_lens, *page_table;
    int64_t num_pages;
    int page_size, max_pages, piece;     // piece: tokens per TMA box
    int B, s_q, H, G, window, sinks;
    float scale, eps;
    int plain, ak_f16;
    const WorkItem* items;
    const int* n_items;
    SchedArgs sa;
    int sched_inline;
    float *o_part, *lse_part;
    void* o;
    int o_dtype;
    float* lse;
    int* status;
};

// Two values as two e4m3 parts each, hi = e4m3(a) and lo = a - hi, a pair packed in 16 bits.  Through fp16, which
// holds a scaled bf16 query exactly down to 2^-17 and has packed conversions; the remainder, at most half a step,
// is exact.
__device__ __forceinline__ void split8(float2 v, uint32_t& hi, uint32_t& lo) {
    const __half2 w = __floats2half2_rn(v.x, v.y);
    const __nv_fp8x2_storage_t h =
        __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(w), __NV_SATFINITE, __NV_E4M3);
    const __half2 r = __hsub2(w, __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
    hi = h;
    lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E4M3);
}

// Four weights (fp16: 11 bits, steps of 2^-24 at the bottom) as hi in e4m3 and a remainder: with kLoUnit in e4m3
// where one operand holds both parts and has one type (STACKED), else in e5m2, fp16's upper byte.  Rounded to
// nearest, half a step of lo is at most 2^-8 of the weight.  Weights below 2^-6, e4m3's least normal value (hi's
// steps are 2^-9 below it), are rounded by the token's dither: for e5m2 0 .. 255 of the byte that is cut off; in
// e4m3 the remainder is then below its normal values too, and one step of 2^-9, (0 .. 255) - 127.5 of 256, is added.
template <bool STACKED>
struct Dither {
    uint32_t bits;           // for two values
    __device__ __forceinline__ explicit Dither(int token) {
        const uint32_t d = ((uint32_t)token * 0x9E3779B1u) >> 24;
        if constexpr (STACKED) {
            const __half2 h = __float2half2_rn(((float)d - 127.5f) * 7.62939453125e-6f);      // 2^-17
            bits = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            bits = d * 0x00010001u;
        }
    }
};
template <bool STACKED>
__device__ __forceinline__ void split_weights(__half2 a, __half2 b, Dither<STACKED> dither, uint32_t& hi, uint32_t& lo) {
    auto part = [&](__half2 w, uint32_t& h) -> uint32_t {
        const __nv_fp8x2_storage_t c =
            __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(w), __NV_SATFINITE, __NV_E4M3);
        const __half2 r = __hsub2(w, __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
        const uint32_t small = __hlt2_mask(w, __float2half2_rn(0.015625f));
        h = c;
        if constexpr (STACKED) {
            const uint32_t d = small & dither.bits;
            const __half2 l = __hfma2(r, __float2half2_rn(kLoUnit), *reinterpret_cast<const __half2*>(&d));
            return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(l), __NV_SATFINITE, __NV_E4M3);
        } else {
            return *reinterpret_cast<const uint32_t*>(&r) + ((small & dither.bits) | (~small & 0x00800080u));
        }
    };
    uint32_t ha, hb;
    const uint32_t la = part(a, ha), lb = part(b, hb);
    hi = ha | (hb << 16);
    lo = STACKED ? la | (lb << 16) : __byte_perm(la, lb, 0x7531);
}

template <int W>
__device__ __forceinline__ void store_codes(uint8_t* at, const uint32_t (&w)[W]) {
    if constexpr (W == 4) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (W == 2) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(at) = w[0];
}

// Sixteen e4m3 codes, NaNs as 0.
__device__ __forceinline__ uint4 finite_e4m3(uint4 v) {
    auto four = [](uint32_t w) { return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); };
    return make_uint4(four(v.x), four(v.y), four(v.z), four(v.w));
}

// Vote and barrier of a softmax group (named barriers 1 ..).
__device__ __forceinline__ bool group_any(int grp, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
        "bar.red.or.pred p, %1, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"(grp + 1), "r"((uint32_t)pred) : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int grp) { asm volatile("bar.sync %0, 128;" ::"r"(grp + 1) : "memory"); }

// Eight rows' values reduced over the 16 lanes of a half warp that hold them: each exchange halves the rows a lane
// still holds (4 + 2 + 1 shuffles and one for the last pair of lanes, not 32).  Lane l of the half gets row
// `half_row(l)`, pairs of lanes the same one.
__device__ __forceinline__ int half_row(int l) { return ((l >> 3) & 1) * 4 + ((l >> 2) & 1) * 2 + ((l >> 1) & 1); }
template <typename F>
__device__ __forceinline__ float half_warp_reduce(const float (&v)[8], int lane, F op) {
    float a[4], b[2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float send = (lane & 8) ? v[u] : v[u + 4], keep = (lane & 8) ? v[u + 4] : v[u];
        a[u] = op(keep, __shfl_xor_sync(0xffffffffu, send, 8));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const float send = (lane & 4) ? a[u] : a[u + 2], keep = (lane & 4) ? a[u + 2] : a[u];
        b[u] = op(keep, __shfl_xor_sync(0xffffffffu, send, 4));
    }
    const float send = (lane & 2) ? b[0] : b[1], keep = (lane & 2) ? b[1] : b[0];
    const float c = op(keep, __shfl_xor_sync(0xffffffffu, send, 2));
    return op(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

// SPANS: a CTA's rows may belong to several query tokens (the others take 3 % longer with its code).
template <int DC, int DR, int ROWS, bool SPANS>
__global__ void __launch_bounds__(96 + 8 * ROWS, 1)
decode_q8_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                 const Q8Params p) {
    using LY = Q8Layout<DC, DR, ROWS>;
    constexpr int NST = LY::kNst, N = LY::kN, KB = LY::kBlocks, NW = 4 * LY::kGroups, NSB = LY::kNsb;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint8_t* sQ = sm;
    uint64_t* bars = (uint64_t*)(sm + LY::kOffMisc);
    uint64_t* full = bars;                   // [NST] tile landed -> logit MMA
    uint64_t* empty = full + NST;            // [NST] output MMA done -> TMA
    uint64_t* pfull = empty + NST;           // [NST] P written -> output MMA (one arrive per softmax warp)
    uint64_t* odone = pfull + NST;           // [NST] output MMA done -> softmax (rescale, epilogue)
    uint64_t* sfull = odone + NST;           // [NSB] logit MMA done -> softmax
    uint64_t* sfree = sfull + NSB;           // [NSB] softmax read S, R -> MMA
    uint64_t* drain = sfree + NSB;           // [2] abort path: an issuer's MMAs in flight are done
    uint32_t* tmem_slot = (uint32_t*)(bars + LY::kNumBars);
    int* abort_flag = (int*)(tmem_slot + 1);
    float* coef_s = (float*)(sm + LY::kOffMisc + 512);   // scale log2e alpha^q x the row's code scale
    float* m_s = coef_s + ROWS;              // running maximum of the logits (integer)
    float* v_s = m_s + ROWS;                 // running maximum of the contributions (integer)
    float* t_s = v_s + ROWS;                 // largest contribution in the tiles whose maxima were formed
    float* f_s = t_s + ROWS;                 // unit of P: kPUnit 2^(m - v)
    float* corr_s = f_s + ROWS;              // rescale factor of O^T in this tile
    float* inv_s = corr_s + ROWS;            // epilogue: 1 / (f l)
    float* red_s = inv_s + ROWS;             // [2 kinds][4 warps][ROWS]

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // warp: uniform
    if (tid == 32) {                                          // beside the plan's loads; its barriers publish it
        for (int i = 0; i < LY::kNumBars; ++i) {
            const bool warps = (&bars[i] >= pfull && &bars[i] < odone) || (&bars[i] >= sfree && &bars[i] < drain);
            mbar_init(&bars[i], warps ? (uint32_t)NW : 1u);
        }
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&tm_lat);
        prefetch_tmap(&tm_rope);
    }
    WorkItem it;
    int seq_len;
    if (p.sched_inline) {
        __shared__ SchedSmem S;
        compute_schedule<true>(p.seq_lens, p.B, p.s_q, p.sa, (int)blockIdx.y, S, p.status, blockIdx.x == 0 && blockIdx.y == 0);
        if ((int)blockIdx.y >= S.n_items) return;
        it = S.item;
        seq_len = S.item_len;
    } else {
        pdl_wait();
        if ((int)blockIdx.y >= *p.n_items) return;
        it = p.items[blockIdx.y];
        seq_len = p.seq_lens[it.b];
        __syncthreads();
    }
    const int b = it.b;
    const int n_rows = p.s_q * p.H;
    const int row0 = blockIdx.x * ROWS;                      // first row (query token x head) of this CTA
    const bool bad = seq_len < 0 || seq_len > p.max_pages * p.page_size;
    const int len = bad ? 0 : seq_len;
    const TileRange tiles(len, p.s_q, p.window, p.sinks, kT);
    const int jt0 = it.tile_begin;
    const int n_t = max(0, min(it.tile_end, tiles.count) - jt0);
    // tokens some row of this CTA sees: [0, len_last) less [sinks, win_first)
    const int i_first = row0 / p.H, i_last = (min(row0 + ROWS, n_rows) - 1) / p.H;
    const int len_last = max(0, len - p.s_q + i_last + 1);
    const int win_first = p.window > 0 ? len - p.s_q + i_first + 1 - p.window : 0;
    // tokens all its query tokens see: those below end_first, less [sinks, win_last)
    const int end_first = len - p.s_q + i_first + 1, win_last = p.window > 0 ? len - p.s_q + i_last + 1 - p.window : 0;

    if (tid == 0 && bad && blockIdx.x == 0) report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
    pdl_wait();
    pdl_trigger();

    // ---- TMA producer (warp 0): the lanes look up the slots of 32 pieces ahead, one loads them ----
    const int n_pieces = kT / p.piece;
    const uint32_t ak_row = p.plain ? 0u : (uint32_t)(p.G * (p.ak_f16 ? 2 : 4));
    const uint32_t piece_bytes = (uint32_t)p.piece * (DC + 2 * DR + 4 + ak_row);
    const int batch = 32 / n_pieces;                          // tiles whose pieces the lanes hold
    int lane_slot = -1;                                       // of this lane's piece; -1: nobody sees it
    int slots[4];                                             // of the current tile
    auto locate_tile = [&](int j) {
        const int k = j % batch;
        if (k == 0) {
            const int jl = j + lane / n_pieces;
            const int t0 = tiles.tile(jt0 + jl) * kT + (lane % n_pieces) * p.piece;
            // a piece without a token that some row sees is not read (its rows are zeroed by the softmax)
            lane_slot = -1;
            if (jl < n_t && t0 < len_last && (t0 < p.sinks || t0 + p.piece > win_first)) {
                const int pg = t0 / p.page_size;
                int64_t page = p.page_table ? (int64_t)p.page_table[(int64_t)b * p.max_pages + pg]
                                            : (int64_t)b * p.max_pages + pg;
                if (page < 0 || page >= p.num_pages) {
                    report(p.status, QKMLA_ERR_DEVICE_BOUNDS);
                    page = 0;
                }
                lane_slot = (int)(page * p.page_size + t0 % p.page_size);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) slots[q] = __shfl_sync(0xffffffffu, lane_slot, k * n_pieces + q);
    };
    auto issue_tile = [&](int j) {                            // one lane
        const int s = j % NST;
        uint8_t* stg = sm + LY::kOffStage + s * LY::kStage;
        uint64_t* bar = &full[s];
        uint32_t n_want = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) n_want += (q < n_pieces && slots[q] >= 0) ? 1u : 0u;
        mbar_arrive_expect_tx(bar, n_want * piece_bytes);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q >= n_pieces || slots[q] < 0) continue;
            const int at = q * p.piece;
            bulk_load(stg + LY::kOffScale + at * 4, p.kv_scale + slots[q], (uint32_t)p.piece * 4, bar);
            if (ak_row)
                bulk_load(stg + LY::kOffAk + at * ak_row, p.ak + (int64_t)slots[q] * ak_row, (uint32_t)p.piece * ak_row, bar);
            tma_load_4d(stg + (at >> 3) * LY::kGroup, &tm_lat, 0, 0, 0, slots[q] >> 3, bar);
            if (!LY::kRopeIn) tma_load_2d(stg + LY::kOffRope + at * LY::kRopeRow, &tm_rope, 0, slots[q], bar);
        }
    };
    auto prefetch_tile = [&]() {                              // one lane
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q >= n_pieces || slots[q] < 0) continue;
            tma_prefetch_4d(&tm_lat, 0, 0, 0, slots[q] >> 3);
            bulk_prefetch(p.kv_scale + slots[q], (uint32_t)p.piece * 4);
            if (ak_row) bulk_prefetch(p.ak + (int64_t)slots[q] * ak_row, (uint32_t)p.piece * ak_row);
        }
    };
    const size_t grow0 = (size_t)b * n_rows + row0;           // first row in the query arrays
    if (warp == 0) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
        if (n_t > 0) {                                        // the others behind the queries' loads
            locate_tile(0);
            if (elect_one()) issue_tile(0);
            __syncwarp();
        }
    } else if (warp >= 3) {
        // ---- prologue: the query rows as hi / lo parts, a warp per row ----
        constexpr int kOwn = ROWS / NW;                       // rows of a warp: their loads go out together
        uint2 raw[kOwn][DC / 128];
        float rv4[kOwn][DR / 32], aq4[kOwn], gq[DR / 32];
#pragma unroll
        for (int k = 0; k < DR / 32; ++k) gq[k] = (p.plain || !p.grq) ? 1.f : p.grq[lane * (DR / 32) + k];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int r = warp - 3 + i * NW;
            const bool ok = row0 + r < n_rows;
            const uint2* src = reinterpret_cast<const uint2*>(p.qt + (grow0 + r) * DC + lane * (DC / 32));
#pragma unroll
            for (int k = 0; k < DC / 128; ++k) raw[i][k] = ok ? src[k] : make_uint2(0u, 0u);
#pragma unroll
            for (int k = 0; k < DR / 32; ++k) rv4[i][k] = ok ? p.qr[(grow0 + r) * DR + lane * (DR / 32) + k] : 0.f;
            aq4[i] = (ok && !p.plain) ? p.aq[grow0 + r] : ok ? 1.f : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int r = warp - 3 + i * NW;
            const float* rv = rv4[i];
            __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < DC / 128; ++k) {
                top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raw[i][k].x)));
                top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raw[i][k].y)));
            }
            float inv;
            const float top = warp_max(fmaxf(__low2float(top2), __high2float(top2)));
            const float sq = e4m3_scale(top, &inv);
            if (isinf(top)) inv = __int_as_float(0x7fffffff);   // no code is infinite: the row becomes NaN, not saturated
            uint32_t hi[DC / 128], lo[DC / 128];              // 4 codes a word
#pragma unroll
            for (int k = 0; k < DC / 128; ++k) {
                const float2 a0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[i][k].x));
                const float2 a1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[i][k].y));
                uint32_t h0, l0, h1, l1;
                split8(make_float2(a0.x * inv, a0.y * inv), h0, l0);
                split8(make_float2(a1.x * inv, a1.y * inv), h1, l1);
                hi[k] = h0 | (h1 << 16);
                lo[k] = l0 | (l1 << 16);
            }
            const int col = lane * (DC / 32), c = col & 127;  // a lane's codes lie within a 16-byte chunk
            const uint32_t h = (uint32_t)r, l = (uint32_t)(r + ROWS), blk = (uint32_t)(col >> 7) * (N * 128);
            store_codes<DC / 128>(sQ + blk + h * 128 + (((c >> 4) ^ (h & 7)) << 4) + (c & 15), hi);
            store_codes<DC / 128>(sQ + blk + l * 128 + (((c >> 4) ^ (l & 7)) << 4) + (c & 15), lo);
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < DR / 32; ++k) ss = fmaf(rv[k], rv[k], ss);
            ss = warp_sum(ss);
            // the RoPE query carries scale log2e: R is the RoPE logit in the exp2 domain
            const float beta = p.scale * kLog2e * (p.plain ? 1.f : rsqrtf(ss * (1.f / DR) + p.eps));
#pragma unroll
            for (int k = 0; k < DR / 32; ++k) {
                const int cr = lane * (DR / 32) + k;
                const float val = rv[k] * gq[k] * beta;
                const __nv_bfloat16 vh = __float2bfloat16_rn(val);
                const __nv_bfloat16 vl = __float2bfloat16_rn(val - __bfloat162float(vh));
                const uint32_t oh = DR == 64 ? sw128_offset(r, cr) : sw64_offset(r, cr);
                const uint32_t ol = DR == 64 ? sw128_offset(r + ROWS, cr) : sw64_offset(r + ROWS, cr);
                *reinterpret_cast<__nv_bfloat16*>(sQ + LY::kQLat + oh) = vh;
                *reinterpret_cast<__nv_bfloat16*>(sQ + LY::kQLat + ol) = vl;
            }
            if (lane == 0) {
                coef_s[r] = p.scale * kLog2e * sq * aq4[i];
                m_s[r] = v_s[r] = t_s[r] = -INFINITY;
                f_s[r] = 0.f;
            }
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ===================== TMA producer =====================
        bool go = true;
        int j = 1;
        for (; j < n_t && go; ++j) {
            locate_tile(j);
            if (j >= NST)
                go = __all_sync(0xffffffffu, wait_bounded(&empty[j % NST], ((j / NST) - 1) & 1, p.status) &&
                                                 !*(volatile int*)abort_flag);
            if (go && elect_one()) issue_tile(j);
            // the next tile into L2 while the ring has no room for it: its load then takes the L2's latency
            // (a stage is held for its load, so the load's latency counts against the ring's three tiles)
            if (j >= NST && (j + 1) % batch && j + 1 < n_t) {
                locate_tile(j + 1);
                if (elect_one()) prefetch_tile();
            }
            __syncwarp();
        }
        // no exit with a copy in flight: on the ordinary path the MMA warp has waited for all of them;
        // an abandoned one is waited for here (one never issued runs into the bound)
        if (!go && lane == 0) {
            *(volatile int*)abort_flag = 1;
            for (int q = max(0, j - 1 - NST); q < j; ++q)
                wait_bounded(&full[q % NST], (q / NST) & 1, p.status, 10000000ull);
        }
    } else if (warp == 1) {
        // ===================== logit MMAs =====================
        if (elect_one()) {
            const uint32_t id_s = idesc_e4m3(kT, N, 0, 0);
            const uint32_t id_r = idesc_bf16(kT, N, 0, 0);
            constexpr uint32_t sw = DR == 64 ? kSwizzle128B : kSwizzle64B, sbo = DR == 64 ? 1024 : 512;
            // descriptors are formed once and moved by constant offsets: the issue must keep up with 65 cycles an MMA
            const uint64_t q_lat = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
            const uint64_t q_rope = smem_desc(smem_u32(sQ) + LY::kQLat, 16, sbo, sw);
            const uint64_t st_lat = smem_desc(smem_u32(sm + LY::kOffStage), 16, LY::kGroup, kSwizzle128B);
            const uint64_t st_rope = smem_desc(smem_u32(sm + LY::kOffStage) + LY::kOffRope, 16, LY::kRopeGroup, sw);
            bool ok = true;
            for (int j = 0; j < n_t; ++j) {
                const int s = j % NST;
                const uint64_t lat = st_lat + (uint64_t)(s * (LY::kStage >> 4)), rope = st_rope + (uint64_t)(s * (LY::kStage >> 4));
                const uint32_t d = tmem + (uint32_t)(j % NSB) * (2 * N);
                // the tile first: once the softmax has read S, nothing but the MMAs is left to do
                ok = wait_bounded(&full[s], (j / NST) & 1, p.status) && !*(volatile int*)abort_flag;
                if (ok && j >= NSB) ok = wait_bounded(&sfree[j % NSB], ((j / NSB) - 1) & 1, p.status);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int blk = 0; blk < KB; ++blk)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8(d, lat + (uint64_t)((blk * 1024 + kk * 32) >> 4), q_lat + (uint64_t)((blk * (N * 128) + kk * 32) >> 4),
                               id_s, (blk > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
                for (int kk = 0; kk < DR / 16; ++kk)
                    mma_bf16(d + N, rope + (uint64_t)(kk * 2), q_rope + (uint64_t)(kk * 2), id_r, kk > 0 ? 1u : 0u);
                mma_commit(&sfull[j % NSB]);
            }
            if (!ok) {                       // no exit with an MMA in flight
                *(volatile int*)abort_flag = 1;
                mma_commit(&drain[0]);
                wait_bounded(&drain[0], 0, p.status);
            }
        }
    } else if (warp == 2) {
        // ===================== output MMAs (a thread of their own: neither issue waits for the other's data) ==========
        if (elect_one()) {
            const uint32_t id_o[2] = {idesc_e4m3(128, LY::kON, 1, 1), idesc_e4m3(128, LY::kON, 1, 1, 1)};   // hi, lo
            // A: a chunk's 128 latents x 32 tokens, MN-major (8-token groups kGroup apart).  B: P, MN-major:
            // a token's codes in as many bytes (swizzle of the same width), 8-token groups kPGroup apart.
            constexpr int PN = LY::kON;
            constexpr uint32_t swp = PN == 128 ? kSwizzle128B : PN == 64 ? kSwizzle64B : kSwizzle32B;
            const uint64_t st_lat = smem_desc(smem_u32(sm + LY::kOffStage), 1024, LY::kGroup, kSwizzle128B);
            const uint64_t st_p = smem_desc(smem_u32(sm + LY::kOffStage) + LY::kOffP, LY::kPGroup, LY::kPGroup, swp);
            bool ok = true;
            for (int j = 0; j < n_t; ++j) {
                const int s = j % NST;
                const uint64_t lat = st_lat + (uint64_t)(s * (LY::kStage >> 4)), pw = st_p + (uint64_t)(s * (LY::kStage >> 4));
                ok = wait_bounded(&pfull[s], (j / NST) & 1, p.status) && !*(volatile int*)abort_flag;
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < KB; ++c)
#pragma unroll
                    for (int kk = 0; kk < kT / 32; ++kk)
#pragma unroll
                        for (int part = 0; part < (LY::kStacked ? 1 : 2); ++part)
                            mma_f8(tmem + LY::kColO + c * PN, lat + (uint64_t)((c * 1024 + kk * 4 * LY::kGroup) >> 4),
                                   pw + (uint64_t)((kk * 4 * LY::kPGroup + part * 8 * PN) >> 4), id_o[part],
                                   (j > 0 || kk > 0 || part > 0) ? 1u : 0u);
                mma_commit(&empty[s]);
                mma_commit(&odone[s]);
            }
            if (!ok) {
                *(volatile int*)abort_flag = 1;
                mma_commit(&drain[1]);
                wait_bounded(&drain[1], 0, p.status);
            }
        }
    } else {
        // ===================== softmax: thread = (token, 8 rows); a group of 4 warps takes 16 rows =====================
        const int sub = warp & 3, grp = (warp - 3) >> 2;
        const uint32_t lane_base = (uint32_t)(32 * sub) << 16;
        // M = 64 accumulator: token t sits in TMEM lane t % 16 of sub-partition t / 16; the two-half load
        // gives lanes 0-15 the first 8 rows of the group, lanes 16-31 the next 8 of the same tokens
        const int tl = 16 * sub + (lane & 15);               // token in the tile
        const int ug = grp * 16;                             // first row of the group
        const int u0 = ug + (lane >> 4) * kHpt;               // first row of this thread
        const int hshift = 31 - __clz(p.H / p.G);            // heads a group: 2, 4, 8 or 16 (H >= 16, G <= 8)
        const int h0 = (row0 + u0) % p.H;                    // its head: kHpt divides H, so the rows share a query token
        const int ak_at = tl * p.G + (h0 >> hshift);         // alpha^k of this token for the first of the rows
        // causal length of these rows (those beyond the last query token, of no one, see what it sees)
        const int n_row = max(0, min(len, len - p.s_q + (row0 + u0) / p.H + 1));
        const int w_row = p.window > 0 ? n_row - p.window : 0;
        // this group's rows in registers, two to a packed pair: -m, unit f, row sums
        constexpr int HP2 = kHpt / 2;
        uint64_t nm2[HP2], f2v[HP2], lsum2[HP2];
        const int settle1 = n_t > (LY::kStacked ? 16 : kSettleFrom1) ? kSettle1 : INT32_MAX, settle2 = n_t > kSettleFrom2 ? kSettle2 : INT32_MAX;
        auto reload = [&]() {
#pragma unroll
            for (int u = 0; u < HP2; ++u) {
                nm2[u] = f2(-m_s[u0 + 2 * u], -m_s[u0 + 2 * u + 1]);
                f2v[u] = f2(f_s[u0 + 2 * u], f_s[u0 + 2 * u + 1]);
            }
        };
#pragma unroll
        for (int u = 0; u < HP2; ++u) lsum2[u] = f2(0.f, 0.f);
        reload();
        bool ok = true;
        for (int j = 0; j < n_t; ++j) {
            const int s = j % NST, sb = j % NSB;
            uint8_t* stg = sm + LY::kOffStage + s * LY::kStage;
            const int t = tiles.tile(jt0 + j) * kT + tl;
            const bool sees = t < n_row && (t < p.sinks || t >= w_row);
            const bool any_sees = t < len_last && (t < p.sinks || t >= win_first);   // some row of the CTA
            const bool masked = !__all_sync(0xffffffffu, sees);
            bool got_s = true;                               // one warp polls, the others sleep at the barrier
            if (((warp - 3) & 3) == 0) got_s = wait_bounded(&sfull[sb], (j / NSB) & 1, p.status);
            group_sync(grp);
            tc_fence_after();
            uint64_t x2[HP2];
            float st_raw;
            {
                uint32_t a[kHpt], c[kHpt], d[kHpt], e[kHpt];
                const uint32_t base = tmem + (uint32_t)sb * (2 * N) + lane_base + ug;
                tmem_ld8x2(base, a);
                tmem_ld8x2(base + ROWS, c);
                tmem_ld8x2(base + N, d);
                tmem_ld8x2(base + N + ROWS, e);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfree[sb]);
                // coefficient x alpha^k s_t of the rows.  A group is 2^SH heads, known to the compiler: with a
                // bound known only at run time the loads became a chain of branches, 2650 cycles a tile
                st_raw = *reinterpret_cast<const float*>(stg + LY::kOffScale + tl * 4);
                uint64_t ca2[HP2];
                auto scale_rows = [&](auto sh, auto f16) {
                    constexpr int SH = decltype(sh)::value;
                    float ak[kHpt];
#pragma unroll
                    for (int u = 0; u < kHpt; ++u)
                        ak[u] = (u & ((1 << SH) - 1)) == 0
                                    ? st_raw * load_alpha<decltype(f16)::value>(stg + LY::kOffAk, ak_at + (u >> SH))
                                    : ak[u & ~((1 << SH) - 1)];
#pragma unroll
                    for (int u = 0; u < kHpt; u += 4) {
                        const float4 cf = *reinterpret_cast<const float4*>(coef_s + u0 + u);
                        ca2[u / 2] = f2_mul(f2(cf.x, cf.y), f2(ak[u], ak[u + 1]));
                        ca2[u / 2 + 1] = f2_mul(f2(cf.z, cf.w), f2(ak[u + 2], ak[u + 3]));
                    }
                };
                using std::integral_constant;
                using yes = integral_constant<bool, true>;
                using no = integral_constant<bool, false>;
                if (p.plain) {
#pragma unroll
                    for (int u = 0; u < kHpt; u += 4) {
                        const float4 cf = *reinterpret_cast<const float4*>(coef_s + u0 + u);
                        ca2[u / 2] = f2_mul(f2(cf.x, cf.y), f2(st_raw, st_raw));
                        ca2[u / 2 + 1] = f2_mul(f2(cf.z, cf.w), f2(st_raw, st_raw));
                    }
                } else if (p.ak_f16) {
                    if (hshift == 4) scale_rows(integral_constant<int, 4>(), yes());
                    else if (hshift == 3) scale_rows(integral_constant<int, 3>(), yes());
                    else if (hshift == 2) scale_rows(integral_constant<int, 2>(), yes());
                    else scale_rows(integral_constant<int, 1>(), yes());
                } else {
                    if (hshift == 4) scale_rows(integral_constant<int, 4>(), no());
                    else if (hshift == 3) scale_rows(integral_constant<int, 3>(), no());
                    else if (hshift == 2) scale_rows(integral_constant<int, 2>(), no());
                    else scale_rows(integral_constant<int, 1>(), no());
                }
#pragma unroll
                for (int u = 0; u < HP2; ++u) {
                    const uint64_t sc = f2_add(f2(__uint_as_float(a[2 * u]), __uint_as_float(a[2 * u + 1])),
                                               f2(__uint_as_float(c[2 * u]), __uint_as_float(c[2 * u + 1])));
                    const uint64_t sr = f2_add(f2(__uint_as_float(d[2 * u]), __uint_as_float(d[2 * u + 1])),
                                               f2(__uint_as_float(e[2 * u]), __uint_as_float(e[2 * u + 1])));
                    x2[u] = f2_fma(ca2[u], sc, sr);
                }
                if (masked && !sees) {
#pragma unroll
                    for (int u = 0; u < HP2; ++u) x2[u] = f2(-INFINITY, -INFINITY);
                }
            }
            const float st = any_sees ? st_raw : 0.f;
            uint64_t e2[HP2], w2[HP2];
            float top_e, top_w;
            // weights e = 2^(x - m) and, in units of the output product, w = e s_t f
            auto weigh = [&]() {
                const uint64_t st2 = f2(st, st);
                top_e = top_w = 0.f;
#pragma unroll
                for (int u = 0; u < HP2; ++u) {
                    const float2 d = f2_unpack(f2_add(x2[u], nm2[u]));
                    float2 e = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                    e2[u] = f2(e.x, e.y);
                    w2[u] = f2_mul(e2[u], f2_mul(st2, f2v[u]));
                    const float2 w = f2_unpack(w2[u]);
                    top_e = fmax3(top_e, e.x, e.y);
                    top_w = fmax3_nan(top_w, w.x, w.y);
                }
                if (masked && !sees) {                       // a row without a token yet has -inf less -inf
#pragma unroll
                    for (int u = 0; u < HP2; ++u) e2[u] = w2[u] = f2(0.f, 0.f);
                    top_w = top_e = 0.f;
                }
            };
            weigh();
            const bool settle = j == settle1 || j == settle2;
            const bool need = !(top_w <= kTopP) || top_e > kTopE || j == 0 || settle;
            if (group_any(grp, need || !got_s)) {
                if (group_any(grp, !got_s)) { ok = false; break; }
                // ---- exact maxima of this tile's logits and contributions, per row ----
                const float ls = st > 0.f ? log2f(st) : -INFINITY;
                float xs[kHpt], vs[kHpt];
#pragma unroll
                for (int u = 0; u < kHpt; ++u) {
                    const float2 xp = f2_unpack(x2[u / 2]);
                    const float xu = (u & 1) ? xp.y : xp.x;
                    xs[u] = xu == xu ? xu : -INFINITY;
                    vs[u] = xs[u] + ls;
                }
                const auto larger = [](float a, float b) { return fmaxf(a, b); };
                const float mx = half_warp_reduce(xs, lane, larger), vx = half_warp_reduce(vs, lane, larger);
                if ((lane & 1) == 0) {
                    red_s[sub * ROWS + u0 + half_row(lane)] = mx;
                    red_s[(4 + sub) * ROWS + u0 + half_row(lane)] = vx;
                }
                group_sync(grp);
                const int gt = tid - 96 - grp * 128;
                if (gt < 16) {
                    const int r = ug + gt;
                    float mx = red_s[r], vx = red_s[4 * ROWS + r];
#pragma unroll
                    for (int q = 1; q < 4; ++q) {
                        mx = fmaxf(mx, red_s[q * ROWS + r]);
                        vx = fmaxf(vx, red_s[(4 + q) * ROWS + r]);
                    }
                    const float m0 = m_s[r], v0 = v_s[r], f0 = f_s[r];
                    t_s[r] = vx = fmaxf(vx, t_s[r]);
                    // binades between the largest contribution and 16: the first tiles' will be exceeded
                    const float room = j >= settle2 ? -3.f : j >= settle1 ? (LY::kStacked || n_t > kSettleMore ? 0.f : 1.f) : v0 == -INFINITY ? 2.f : 1.f;
                    const float m1 = mx > m0 + 4.f ? ceilf(mx) : m0;
                    const float v1 = vx > v0 + fmaxf(2.f, 1.f - room) || (settle && vx > -INFINITY) ? ceilf(vx) + room : v0;
                    const float cm = m0 == -INFINITY ? 0.f : exp2f(m0 - m1);       // of the row sums
                    // nothing to add up yet (no visible token, or latents of zeros, whose scale is 0): with the largest
                    // unit the first contribution, whatever its tile, is above kTopP and sets it
                    const float f1 = kPUnit * exp2f(v1 == -INFINITY ? 122.f : fminf(fmaxf(m1 - v1, -126.f), 122.f));
                    m_s[r] = m1;
                    v_s[r] = v1;
                    f_s[r] = f1;
                    red_s[r] = cm;
                    corr_s[r] = f0 > 0.f ? cm * f1 / f0 : 0.f;                     // of O^T; nothing there yet: 0
                }
                group_sync(grp);
                if (j > 0) {
                    const bool got_o = wait_bounded(&odone[(j - 1) % NST], ((j - 1) / NST) & 1, p.status);
                    if (group_any(grp, !got_o)) { ok = false; break; }
                    tc_fence_after();
                    bool moved = false;
#pragma unroll
                    for (int u = 0; u < 16; ++u) moved = moved || corr_s[ug + u] != 1.f;
                    if (moved) {
#pragma unroll 1
                        for (int c = 0; c < KB * (LY::kStacked ? 2 : 1); ++c) {     // chunks (x hi, lo)
                            uint32_t v[16];
                            const uint32_t ta = tmem + LY::kColO + c * ROWS + ug + lane_base;
                            tmem_ld16(ta, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; ++u) {
                                const float cr = corr_s[ug + u];
                                v[u] = cr == 0.f ? 0u : __float_as_uint(__uint_as_float(v[u]) * cr);
                            }
                            tmem_st16(ta, v);
                        }
                        tmem_wait_st();
                    }
                }
#pragma unroll
                for (int u = 0; u < HP2; ++u)
                    lsum2[u] = f2_mul(lsum2[u], f2(red_s[u0 + 2 * u], red_s[u0 + 2 * u + 1]));
                reload();
                weigh();
#pragma unroll
                for (int u = 0; u < HP2; ++u) {              // s_t f beyond fp32 beside e = 0: no weight, not NaN
                    const float2 e = f2_unpack(e2[u]), w = f2_unpack(w2[u]);
                    w2[u] = f2(e.x == 0.f ? 0.f : w.x, e.y == 0.f ? 0.f : w.y);
                }
                group_sync(grp);                             // red_s, corr_s are read
            }
            const Dither<LY::kStacked> dither(t);
            uint32_t hi[kHpt / 4], lo[kHpt / 4];
#pragma unroll
            for (int u = 0; u < HP2; u += 2) {
                const float2 wa = f2_unpack(w2[u]), wb = f2_unpack(w2[u + 1]);
                split_weights(__floats2half2_rn(wa.x, wa.y), __floats2half2_rn(wb.x, wb.y), dither, hi[u / 2], lo[u / 2]);
                lsum2[u] = f2_add(lsum2[u], e2[u]);
                lsum2[u + 1] = f2_add(lsum2[u + 1], e2[u + 1]);
            }
            // P row of this token: 8 codes of hi at u0 and of lo at ROWS + u0 (one operand) or at u0 of the next
            // operand, 16-byte chunks XOR-swizzled (rows of 128, 64, 32 bytes: by token, token / 2, token / 4)
            constexpr int PN = LY::kON;
            uint8_t* pr = stg + LY::kOffP + (tl >> 3) * LY::kPGroup + (tl & 7) * PN + (u0 & 15);
            const uint32_t xr = PN == 128 ? tl & 7 : PN == 64 ? (tl >> 1) & 3 : (tl >> 2) & 1;
            const uint32_t chi = (uint32_t)u0 >> 4, clo = LY::kStacked ? (uint32_t)(ROWS + u0) >> 4 : chi;
            *reinterpret_cast<uint2*>(pr + ((chi ^ xr) << 4)) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(pr + (LY::kStacked ? 0 : 8 * PN) + ((clo ^ xr) << 4)) = make_uint2(lo[0], lo[1]);
            // a token no row sees: its latents (stale or never loaded) must not reach the output MMA as NaN; a token
            // that only some of the CTA's query tokens see: its NaNs must not reach the others' rows as 0 x NaN (in
            // the rows that see it the logit is NaN)
            if (!any_sees || (SPANS && (t >= end_first || (t >= p.sinks && t < win_last)))) {
                constexpr int kShare = 2 * LY::kGroups;      // threads of a token
                for (int c = 2 * grp + (lane >> 4); c < 8 * KB; c += kShare) {
                    uint4* at = reinterpret_cast<uint4*>(stg + (tl >> 3) * LY::kGroup + (c >> 3) * 1024 + (tl & 7) * 128 +
                                                         (((c & 7) ^ (tl & 7)) << 4));
                    *at = SPANS && any_sees ? finite_e4m3(*at) : make_uint4(0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[s]);
        }
        if (!ok) *(volatile int*)abort_flag = 1;
        // ---- epilogue: row sums over the tokens, then O^T / (f l) ----
        float ls[kHpt];
#pragma unroll
        for (int u = 0; u < HP2; ++u) {
            const float2 l2 = f2_unpack(lsum2[u]);
            ls[2 * u] = l2.x;
            ls[2 * u + 1] = l2.y;
        }
        const float sum = half_warp_reduce(ls, lane, [](float a, float b) { return a + b; });
        if ((lane & 1) == 0) red_s[sub * ROWS + u0 + half_row(lane)] = sum;
        const bool got_last = (ok && n_t > 0) ? wait_bounded(&odone[(n_t - 1) % NST], ((n_t - 1) / NST) & 1, p.status) : ok;
        if (group_any(grp, !got_last)) *(volatile int*)abort_flag = 1;
        tc_fence_after();
        const int gt = tid - 96 - grp * 128;
        if (gt < 16) {
            const int r = ug + gt;
            const float l = (red_s[r] + red_s[ROWS + r]) + (red_s[2 * ROWS + r] + red_s[3 * ROWS + r]);
            const float lse = l > 0.f ? (m_s[r] + log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
            inv_s[r] = l == 0.f ? 0.f : 1.f / f_s[r] / l;
            if (row0 + r < n_rows) {
                if (it.part >= 0) p.lse_part[(size_t)it.part * n_rows + row0 + r] = lse;
                else if (p.lse) p.lse[grow0 + r] = lse;
            }
        }
        group_sync(grp);
        float inv[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) inv[u] = inv_s[ug + u];
        const int n_out = n_rows - row0 - ug;                 // rows of the group that exist
        const size_t at = (it.part >= 0 ? (size_t)it.part * n_rows + row0 + ug : grow0 + ug) * DC + 32 * sub + lane;
        float* const dst_f = it.part >= 0 ? p.o_part + at : (float*)p.o + at;
        __nv_bfloat16* const dst_h = (__nv_bfloat16*)p.o + at;
        const bool f32 = it.part >= 0 || p.o_dtype == QKMLA_F32;
#pragma unroll 1
        for (int c = 0; c < KB; ++c) {
            uint32_t a[16];
            float val[16];
            if (n_t > 0) {
                tmem_ld16(tmem + LY::kColO + c * LY::kON + ug + lane_base, a);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u) val[u] = __uint_as_float(a[u]);
                if constexpr (LY::kStacked) {
                    tmem_ld16(tmem + LY::kColO + c * LY::kON + ROWS + ug + lane_base, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 16; ++u) val[u] = fmaf(__uint_as_float(a[u]), 1.f / kLoUnit, val[u]);
                }
#pragma unroll
                for (int u = 0; u < 16; ++u) val[u] = inv[u] == 0.f ? 0.f : val[u] * inv[u];
            } else {
#pragma unroll
                for (int u = 0; u < 16; ++u) val[u] = 0.f;
            }
            if (f32) {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    if (u < n_out) dst_f[c * 128 + u * DC] = val[u];
            } else {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    if (u < n_out) dst_h[c * 128 + u * DC] = __float2bfloat16_rn(val[u]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Cache rows as a 4-D tensor: 128-byte blocks of a row, 8 rows, the blocks, the groups of 8 rows -- a box
// of it lands in shared memory as the atoms the tensor core reads.
bool make_row_map(CUtensorMap* m, const void* base, int64_t rows, int64_t pitch, int blocks, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {128, 8, (cuuint64_t)blocks, (cuuint64_t)(rows / 8)};
    cuuint64_t strides[3] = {(cuuint64_t)pitch, 128, (cuuint64_t)(8 * pitch)};
    cuuint32_t box[4] = {128, 8, (cuuint32_t)blocks, (cuuint32_t)(box_rows / 8)};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The RoPE key of rows whose key is not a block of its own (d_r = 32: 64 bytes a row).
bool make_rope_map(CUtensorMap* m, const void* base, int64_t rows, int64_t pitch, int d_r, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)d_r, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {(cuuint32_t)d_r, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows per CTA: as many as there are, to 64.
int q8_rows(const qkmla_decode_args* a) {
    const int n = a->s_q * a->H;
    return n <= 16 ? 16 : n <= 32 ? 32 : 64;
}
int q8_row_blocks(const qkmla_decode_args* a) {
    const int r = q8_rows(a);
    return (a->s_q * a->H + r - 1) / r;
}

template <int DC, int DR, int ROWS>
int launch_q8(const Q8Params& q, const CUtensorMap& lat, const CUtensorMap& rope, dim3 grid, cudaStream_t s) {
    const bool spans = q.s_q > 1 && q.H % ROWS != 0;          // 16 rows are at most one query token's
    auto k = ROWS > 16 && spans ? decode_q8_kernel<DC, DR, ROWS, (ROWS > 16)> : decode_q8_kernel<DC, DR, ROWS, false>;
    constexpr int bytes = Q8Layout<DC, DR, ROWS>::kBytes;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return QKMLA_ERR_CUDA;
    return launch_pdl(k, grid, dim3(Q8Layout<DC, DR, ROWS>::kThreads), bytes, s, lat, rope, q) == cudaSuccess
               ? QKMLA_OK
               : QKMLA_ERR_CUDA;
}

}  // namespace

// 8-bit cache shapes of the tensor-core kernel.  A thread's 8 rows share a query
// token when 8 divides H; a tile is made of whole pages or a page of whole tiles.
bool q8_tc_supported(const qkmla_decode_args* a, const DecodeExt& x) {
    if (a->cache_dtype != QKMLA_E4M3) return false;
    if (!((a->d_c == 512 && a->d_r == 64) || (a->d_c == 256 && (a->d_r == 32 || a->d_r == 64)) ||
          (a->d_c == 128 && (a->d_r == 32 || a->d_r == 64))))
        return false;
    if (a->H % 16 || a->G > kMaxG || a->B > kMaxB) return false;
    if (a->page_size % 16 || (a->page_size < kT ? kT % a->page_size : a->page_size % kT)) return false;
    if (a->num_slots > 2147483647LL) return false;                // TMA row coordinates are 32-bit
    if (((uintptr_t)a->kv_cache % 16) || ((uintptr_t)a->q_tilde % 16) || ((uintptr_t)a->o % 16) ||
        ((uintptr_t)x.kv_scale % 16))
        return false;
    return (a->flags & QKMLA_FLAG_PLAIN_MLA) || ((uintptr_t)a->ak_cache % 16) == 0;
}

size_t q8_tc_workspace(const qkmla_decode_args* a, int sms) {
    return split_scratch(a, q8_row_blocks(a), sms, nullptr).bytes;
}

int launch_decode_q8(const qkmla_decode_args* a, const DecodeExt& x, cudaStream_t s) {
    const int sms = device_sm_count();
    const int n_rb = q8_row_blocks(a);
    const SplitScratch w = split_scratch(a, n_rb, sms, a->workspace);
    SchedArgs sa;
    sa.max_len = a->max_pages * a->page_size;
    sa.n_rb = n_rb;
    sa.sms = sms;
    sa.min_tokens = kMinItemTokens;
    sa.tile = kT;
    sa.fixed_splits = a->num_splits;
    sa.min_len = 0;
    sa.window = x.window;
    sa.sinks = x.sinks;
    sa.chunks = never_splits(a, x) ? 0 : chunks_of(a, x, sa);
    const int sched_inline = sched_in_kernel(a) ? 1 : 0;
    if (!sched_inline && launch_sched(a, sa, w, s) != QKMLA_OK) return QKMLA_ERR_CUDA;

    Q8Params q;
    q.qt = (const __nv_bfloat16*)a->q_tilde;
    q.aq = a->alpha_q;
    q.qr = a->q_rope;
    q.grq = a->gamma_rope_q;
    q.ak = (const uint8_t*)a->ak_cache;
    q.kv_scale = x.kv_scale;
    q.seq_lens = a->seq_lens;
    q.page_table = a->page_table;
    q.num_pages = a->num_slots / a->page_size;
    q.page_size = a->page_size;
    q.max_pages = a->max_pages;
    q.piece = std::min(a->page_size, kT);
    q.B = a->B; q.s_q = a->s_q; q.H = a->H; q.G = a->G;
    q.window = x.window;
    q.sinks = x.sinks;
    q.scale = a->softmax_scale;
    q.eps = a->eps;
    q.plain = (a->flags & QKMLA_FLAG_PLAIN_MLA) ? 1 : 0;
    q.ak_f16 = (a->flags & QKMLA_FLAG_ALPHA_F16) ? 1 : 0;
    q.items = w.items;
    q.n_items = w.n_items;
    q.sa = sa;
    q.sched_inline = sched_inline;
    q.o_part = w.o_part;
    q.lse_part = w.lse_part;
    q.o = a->o;
    q.o_dtype = a->o_dtype;
    q.lse = a->lse;
    q.status = device_status_ptr();

    const int64_t pitch = a->d_c + 2 * a->d_r;
    CUtensorMap lat, rope;
    if (!make_row_map(&lat, a->kv_cache, a->num_slots, pitch, a->d_c / 128 + (a->d_r == 64 ? 1 : 0), q.piece)) return QKMLA_ERR_CUDA;
    if (a->d_r == 64) rope = lat;
    else if (!make_rope_map(&rope, (const uint8_t*)a->kv_cache + a->d_c, a->num_slots, pitch, a->d_r, q.piece))
        return QKMLA_ERR_CUDA;
    const dim3 grid(n_rb, w.max_items);
    const int rows = q8_rows(a);
    auto by_rows = [&](auto dc, auto dr) {
        constexpr int DC = decltype(dc)::value, DR = decltype(dr)::value;
        return rows == 16   ? launch_q8<DC, DR, 16>(q, lat, rope, grid, s)
               : rows == 32 ? launch_q8<DC, DR, 32>(q, lat, rope, grid, s)
                            : launch_q8<DC, DR, 64>(q, lat, rope, grid, s);
    };
    using std::integral_constant;
    using d32 = integral_constant<int, 32>;
    using d64 = integral_constant<int, 64>;
    const int rc = a->d_c == 512   ? by_rows(integral_constant<int, 512>(), d64())
                   : a->d_c == 256 ? (a->d_r == 32 ? by_rows(integral_constant<int, 256>(), d32())
                                                   : by_rows(integral_constant<int, 256>(), d64()))
                   : a->d_r == 32  ? by_rows(integral_constant<int, 128>(), d32())
                                   : by_rows(integral_constant<int, 128>(), d64());
    if (rc != QKMLA_OK || never_splits(a, x)) return rc;
    return launch_combine_var(a, sa, w, s);
}

}  // namespace qkmla
