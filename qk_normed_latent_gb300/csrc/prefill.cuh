// What the kernels of qkmla_prefill share: sizes, the workspace and the plan of the attention's work.
//
// A call runs three kernels.  prefill_expand_kernel recovers keys and values of the cached tokens (its last block
// makes the plan), prefill_attend_kernel normalises the queries and attends, prefill_join_kernel joins the rows
// whose tokens were cut between two CTAs.
//
// Everything a tensor-core product reads is written in 16 KB blocks of 128 rows x 64 fp16 values, as it lies in
// shared memory (rows of 128 bytes, 128-byte swizzle), so that one contiguous bulk copy brings it in and no tensor
// map is made.
#pragma once

#include "common.cuh"
#include "decode_common.cuh"
#include "tc_ptx.cuh"

namespace qkmla {
namespace pf {

constexpr int kTile = 128;                 // tokens of a tile
constexpr int kRowsQ = 256;                // query rows (tokens x heads of a unit) of a tile: two halves of 128
constexpr int kBlock = 16384;              // bytes of a block of 128 x 64 values
constexpr int kMaxE = 40;                  // largest exponent of a tile's values
constexpr int kNone = -1000, kBad = 1000;  // exponents of an all-zero and of a not finite token
// Cost of starting on a query tile, in tiles of tokens (17 rows over 333 tokens, ragged chunks at 16 heads and at 128: 28.6, 107.8 and
// 190 us; with 1 35.1, 107.4 and 191, with 8 28.3, 114.5 and 199).
constexpr int kCostStart = 4;
constexpr int kMinPiece = 2;               // no piece of a cut query tile has fewer tiles of tokens (ragged chunks 190 us, with 1 191, with 4 189)
// Pieces of work listed, and their queries normalised, ahead: with 2 a short piece ends before the next one's queries are
// there (1024 queries over 16000 tokens 829 us, with 4 812; 4 prompts of 4096 2015 and 2000; 6 no better than 4).
constexpr int kAhead = 4;
constexpr int kMaxCtas = 256;
constexpr int kMinShare = 6;               // nor a CTA fewer units of cost (17 rows over 333 tokens 28.6 us, with 2 28.5, with 16 47.3)

struct Params {
    // the caller's
    const void *q, *q_rope;
    int64_t q_row, q_head, qr_row, qr_head;
    const float *gamma_q, *gamma_k, *gamma_rope;
    const uint8_t* weights;
    const uint8_t* kv;
    const float* kv_scale;
    const void* ak;
    const int32_t *chunk_start, *seq_lens, *page_table;
    int64_t num_pages;
    int page_size, max_pages;
    int B, rows, H, G, Gv, d_c, d_h, d_r, d_v;
    float scale_log2, eps;
    int window, sinks;
    int ak_f16, q_bf16, o_f32;
    int64_t total_tokens;
    void* o;
    float* lse;
    // derived
    int units;                             // heads with a key and a value matrix in common: max(G, G_v) units
    int hp, hp_log;                        // heads of a unit, a power of two
    int tq;                                // query tokens of a tile: 256 / hp
    int nq;                                // slots of query tiles: rows / tq + B
    int max_tiles;                         // total_tokens / 128 + B
    int ctas;                              // of the attention kernel
    int deep;                              // places a CTA: units nq / ctas, rounded up
    // the workspace
    int4* seq;                             // [B][2]: {length, first tile, first row, rows}, {tiles left out behind its head, -}
    int4* qinfo;                           // [nq][2]: {b, first query, tiles, head tiles}, {gap, length of the first query, queries, -}
    int64_t* pre;                          // [ctas deep + 1]: cost of the places ahead
    int4* cuts;                            // [ctas + 1]: where each CTA's share starts
    int* tinfo;                            // [max_tiles]: TileScale::packed()
    uint8_t *krope, *kc, *v;               // blocks: [tile], [tile][G][d_h / 64], [tile][G_v][d_v / 64]
    uint8_t* qs;                           // [cta][kAhead][half][d_h / 64 + 1]: the normalised queries of a CTA's next pieces
    float* part_o;                         // [2 ctas][256][d_v]
    float2* part_ml;                       // [2 ctas][256]: reference and sum
    int* status;
};

// The packed weights: fp16 blocks of 64 output columns x 64 latents, [N-tile][d_c / 64][2 or 4 blocks of columns], after a
// table of the power of two of each matrix.
__host__ __device__ inline int column_blocks(int G, int Gv, int d_h, int d_v) { return G * (d_h / 64) + Gv * (d_v / 64); }
__host__ __device__ inline int blocks_per_tile(int d_c) { return d_c > 256 ? 4 : 2; }    // column blocks of an N-tile
__host__ __device__ inline int n_tiles(int G, int Gv, int d_h, int d_v, int d_c) {
    return (column_blocks(G, Gv, d_h, d_v) + blocks_per_tile(d_c) - 1) / blocks_per_tile(d_c);
}
constexpr size_t kWeightTable = 4096;      // int32 exponents of up to 1024 matrices

// Token tiles of a sequence that its rows see: those below `head` and those from head + gap on (all of them without a
// window, none for a sequence without rows or with a bad length).  The workspace holds these alone, one sequence's
// behind the other's.
struct Needed { int tiles, head, gap; };
__device__ __forceinline__ Needed needed(const Params& p, int len, int rows) {
    if (len < 0 || len > (int64_t)p.max_pages * p.page_size || rows <= 0) return Needed{0, 0, 0};
    const int total = (len + kTile - 1) / kTile;
    const int64_t lo = (int64_t)len - rows + 1 - p.window;              // the first row's window starts here
    if (p.window > 0 && lo > 0) {
        const int from = (int)(lo / kTile), head = (int)((min((int64_t)p.sinks, lo) + kTile - 1) / kTile);
        if (from > head) return Needed{total - (from - head), head, from - head};
    }
    return Needed{total, total, 0};
}

// First slot of a sequence's query tiles: its rows start at chunk_start[b], and rounding up for each of the
// b sequences ahead takes at most b slots, so ranges never meet and need no sum over the sequences.
__device__ __forceinline__ int first_slot(int row, int b, int tq) { return row / tq + b; }

// The list of all work.  Query tiles in their own order -- by unit, sequence and row -- are dealt out to the CTAs in turn,
// and the list is one CTA's hand after the other's: place m = c deep + i holds the tile i ctas + c.  An even share of the
// list is then about a hand, and at any time the CTAs work on neighbouring tiles, whose keys and values the L2 holds (a
// CTA on neighbouring tiles of its own has all units' going at once: 2.6 times the traffic to memory on whole prompts).
__device__ __forceinline__ bool tile_of_place(const Params& p, int m, int& u, int& j) {
    const int c = m / p.deep, n = (m - c * p.deep) * p.ctas + c;
    u = n / p.nq;
    j = n - u * p.nq;
    return u < p.units;
}

// A place, and a tile `t` of tokens of it out of nt.
struct Place {
    int m, t, nt;
    __device__ __forceinline__ bool same(const Place& o) const { return m == o.m && t == o.t; }
    __device__ __forceinline__ bool inside() const { return t > 0 && t < nt; }
};
// A cut that would leave a piece of fewer than kMinPiece tiles moves to the query tile's start or end.
__device__ __forceinline__ Place place_at(const Params& p, int m, int64_t x) {
    Place r;
    r.m = m;
    const int64_t at = p.pre[m];
    r.nt = (int)(p.pre[m + 1] - at) - kCostStart;
    const int t = (int)(x - at) - kCostStart;
    r.t = t < kMinPiece ? 0 : r.nt - t < kMinPiece ? r.nt : t;
    return r;
}

// The place of cost x, 0 <= x <= all, all > 0 (for x = all the end of the last query tile): whole warp.
__device__ __forceinline__ Place place_of(const Params& p, int64_t x, int64_t all) {
    const bool end = x == all;
    if (end) --x;
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.ctas * p.deep;                       // the last m in [lo, lo + n) with pre[m] <= x
#pragma unroll 1
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && p.pre[lo + lane * step] <= x;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = 31 - __clz(m | 1u);
        n = min(step, n - k * step);
        lo += k * step;
    }
    Place r = place_at(p, lo, x);
    if (end) r.t = r.nt;
    return r;
}

// CTAs that share the work: no more than leave each kMinShare.
__device__ __forceinline__ int sharing(const Params& p, int64_t all) {
    const int64_t n = all / kMinShare;
    return n < 1 ? 1 : n < p.ctas ? (int)n : p.ctas;
}
__device__ __forceinline__ int64_t share_start(int64_t all, int n, int c) { return all / n * c + all % n * c / n; }

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^e as an exact float, e in [-126, 127]
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// How a tile's values are held, from the largest and the least exponent of its tokens' latents (zeros left out): as 2^-e of
// themselves, in fp16 or, where that would not hold them beside one another, bf16.  A row's softmax reference follows the
// tile that moves it, of weight 2^e there; a row may not see the tile's largest token, or give it no weight, and a reference
// too high takes bits from the weights of all other tiles.  So the reference is set `drop` lower, e - drop the least
// exponent: bf16 has the range to take that one as e; fp16's values grow by up to 2^4 (2^11, the sum of 512 products of
// numbers below 2, becomes 2^15), and its weights give up to 2^8 of their own room above 2^7.
struct TileScale {
    int e, drop;
    bool bf;
    __device__ __forceinline__ TileScale(int hi, int lo) {
        const int spread = hi - lo;
        bf = hi != kNone && (spread > 12 || hi > kMaxE || hi < -kMaxE);
        if (hi == kNone) e = -kMaxE;                       // zeros are of no size that others are measured by
        else if (bf) e = min(max(lo, max(hi - 80, -kMaxE)), kMaxE);      // (values then stay below 2^91, or as large as they are)
        else e = hi - min(spread, 4);
        drop = bf || hi == kNone ? 0 : spread - min(spread, 4);
    }
    // [e + 64 | bf << 8 | drop << 9]
    __device__ __forceinline__ int packed() const { return (e + 64) | (bf ? 256 : 0) | drop << 9; }
};

// Every wait ends by itself, after kSpins tries (each of 50 ns or more); a warp that gives up says so and leaves, and the
// others' waits end likewise.  (Named barriers cannot be used where a thread may have given up.)  Small on purpose: beyond
// some 64 KB of code the instruction cache misses and every warp slows down to 5 cycles an instruction and more.
constexpr uint32_t kSpins = 1u << 22;
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, int* fail) {
    uint32_t i = 0;
#pragma unroll 1
    while (!tc::mbar_try_wait(bar, parity))
        if (++i == kSpins) {
            *(volatile int*)fail = 1;
            return false;
        }
    return true;
}

// The same for a wait that may last as long as a whole query tile's work: it ends when another warp gives up, too.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* fail) {
    uint32_t i = 0;
#pragma unroll 1
    while (!tc::mbar_try_wait(bar, parity))
        if (++i == 1u << 28 || *(volatile int*)fail) {
            *(volatile int*)fail = 1;
            return false;
        }
    return true;
}

// Descriptors as their low word (address and leading offset) and a high word common to all (rows of 128 bytes, 8-row
// groups 1024 apart): the products then take 8 machine instructions each where 64-bit descriptors took 16, and the issue's
// code half the room.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | tc::kSwizzle128B << 29;
__device__ __forceinline__ uint32_t desc_low(const void* at, uint32_t lbo) { return (tc::smem_u32(at) >> 4) | lbo >> 4 << 16; }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(acc)
        : "memory");
}
// A out of TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
        ::"r"(d), "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&a)[4], const uint32_t (&b)[4]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]),
                 "r"(b[1]), "r"(b[2]), "r"(b[3])
                 : "memory");
}

// Four rows a quad of lanes, four pieces of 32 bytes a row: from piece k of the lane's own row in h[k] to piece lane % 4 of
// row k of the quad.  A store of a row a lane touches 32 lines an instruction, and each costs a cycle of the data path that
// the tensor core's operands come through; a quad's four lanes then write one whole line.
__device__ __forceinline__ void quad_transpose(uint32_t (&h)[4][8], int lane) {
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & bit) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t r = __shfl_xor_sync(0xffffffffu, up ? h[k][i] : h[k | bit][i], bit);
                if (up) h[k][i] = r;
                else h[k | bit][i] = r;
            }
        }
    }
}

int launch_expand(const Params& p, bool q8, cudaStream_t s);
int launch_attend(const Params& p, cudaStream_t s);

}  // namespace pf
}  // namespace qkmla
