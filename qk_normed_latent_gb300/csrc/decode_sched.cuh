// Split-KV schedule computed inside the kernels that need it (decode, combine).
//
// Every CTA derives the same plan from seq_lens, so no separate scheduler launch
// (and no kernel boundary) sits between the previous kernel and the decode:
//   * tiles per sequence tb_b = ceil(L_b / tile), less those outside a window;
//   * tiles per work item tpi: the longest sequence when that is within 25 % of
//     an even share of the GPU (s_total * n_rb / sms), else that share rounded
//     up; at least min_tokens worth of tiles;
//   * a sequence splits into ns_b = ceil(tb_b / tpi) items (or the caller's
//     fixed split count), of per = ceil(tb_b / ns_b) tiles each;
//   * items are numbered by sequence, longest first (ties by index), so the
//     work that bounds the tail starts first; an item's index is also the index
//     of its partial output when its sequence is split.
// A plan of chunks takes the place of the last two points where they make more
// items than the GPU takes at once and an even share is kChunkTiles or more: a
// sequence is cut into chunks of 1.05 shares and a remainder (spread over the
// chunks if below min_tokens); all chunks start first, then the remainders, longest
// first.  Equal parts of about a share leave nothing short to fill up the second
// wave: 32 sequences of 512-32k tokens, two query tokens, 8-bit cache, 208 us
// against 172 (179 since small weights keep their sum); windowed, bf16, 227 against 199.  (Chunks of 0.9-1.15 shares and the
// best of 8 lengths of equal parts are behind in a model of the plan.)  It costs
// other calls up to 0.4 us.  Only qkmla_decode_ext's calls use it: the others keep
// their results bit for bit.
// Ranking costs B^2 / 32 / warps votes, so this path serves batches of up to
// kMaxBSched sequences; larger batches use the scheduler kernel.
#pragma once

#include "decode_common.cuh"

namespace qkmla {
namespace dec {

constexpr int kMaxBSched = 128;

struct SchedSmem {
    int len[kMaxBSched];       // seq_lens[b] as read
    int tb[kMaxBSched];        // tiles of sequence b
    int ns[kMaxBSched];        // items of sequence b
    int base[kMaxBSched];      // first partial output of sequence b
    int by_rank[kMaxBSched];   // sequence at rank k
    int split[kMaxBSched];     // the split sequences (ns > 1), in rank order
    int n_items, n_split;
    WorkItem item;             // the caller's item and its sequence's length
    int item_len;
};

// Block-wide: every thread of the CTA calls it; on return `S` holds the plan, with item number `item` where it
// exists (item < S.n_items).
// Sequences with an invalid length get no tiles (and a status report when
// `report_errors`).  With SPLITS_ONLY (the combine kernel) a plan without a split
// sequence ends as soon as that is known: n_split is 0 and nothing else is set.
// CHUNKS: the kernel serves calls whose plan may be one of chunks.
template <bool CHUNKS, bool SPLITS_ONLY = false>
__device__ __forceinline__ void compute_schedule(const int32_t* __restrict__ seq_lens, int B, int s_q,
                                                 const SchedArgs& a, int item, SchedSmem& S, int* status,
                                                 bool report_errors) {
    constexpr int K = kMaxBSched / 32;
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    for (int b = tid; b < B; b += nt) {
        const int L = __ldcg(seq_lens + b);   // through L2: the lengths may change between calls
        S.len[b] = L;
        int tl = 0;
        if (L < a.min_len || L > a.max_len) {
            if (report_errors) report(status, QKMLA_ERR_DEVICE_BOUNDS);
        } else {
            tl = TileRange(L, s_q, a.window, a.sinks, a.tile).count;
        }
        S.tb[b] = tl;
    }
    __syncthreads();
    // every warp holds all tile counts, sequence 32 i + lane in tb[i], and forms the totals and its share of the
    // ranks with votes: no further barrier until the ranks are written
    int tb[K], tot = 0, m = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        tb[i] = 32 * i + lane < B ? S.tb[32 * i + lane] : -1;
        tot += max(tb[i], 0);
        m = max(m, tb[i]);
    }
    tot = __reduce_add_sync(0xffffffffu, tot);
    m = __reduce_max_sync(0xffffffffu, m);
    const float ideal = (float)tot * a.n_rb / (float)a.sms;
    const int least = a.min_tokens / a.tile;
    const int tpi = max(max((float)m <= 1.25f * ideal ? m : (int)ceilf(ideal), least), 1);
    int chunk = 0;                              // tiles of a chunk; 0: equal parts
    if (CHUNKS && a.chunks && ideal >= (float)kChunkTiles) {
        int items = 0;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (tb[i] >= 0) items += max(1, (int)((uint32_t)(tb[i] + tpi - 1) / (uint32_t)tpi));
        if (__reduce_add_sync(0xffffffffu, items) * a.n_rb > a.sms) chunk = (int)ceilf(1.05f * ideal);
    }
    // chunks of a sequence and its remainder (0: none, or spread over the chunks)
    auto cut = [&](int tiles, int& full, int& rest) {
        full = (int)((uint32_t)tiles / (uint32_t)chunk);
        rest = tiles - full * chunk;
        if (full > 0 && rest < least) rest = 0;
    };
    if constexpr (SPLITS_ONLY) {
        if (a.fixed_splits == 0 && m <= (CHUNKS && chunk ? chunk : tpi)) {      // uniform
            if (tid == 0) S.n_split = 0;
            __syncthreads();
            return;
        }
    }
    if (CHUNKS && chunk) {                      // ranked by their remainders
#pragma unroll
        for (int i = 0; i < K; ++i) {
            int full;
            if (tb[i] >= 0) cut(tb[i], full, tb[i]);
        }
    }
    for (int b = warp; b < B; b += nw) {
        int mine = S.tb[b], full;
        if (CHUNKS && chunk) cut(mine, full, mine);
        int rk = 0;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (32 * i < B)
                rk += __popc(__ballot_sync(0xffffffffu, tb[i] > mine || (tb[i] == mine && 32 * i + lane < b)));
        if (lane == 0) S.by_rank[rk] = b;
    }
    __syncthreads();
    // exclusive prefix of the item counts in rank order (one warp, B <= 128: four ranks a lane)
    if (warp == 0) {
        int v[K], sp[K], fl[K];                 // parts, split or not, parts among the first items
        int run = 0, nsp = 0, nfl = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int k = lane * K + i;
            v[i] = fl[i] = 0;
            if (k < B) {
                const int b = S.by_rank[k], tiles = S.tb[b];
                if (CHUNKS && chunk) {
                    int rest;
                    cut(tiles, fl[i], rest);
                    if (tiles == 0) rest = 1;   // an item of its own, without a tile
                    v[i] = fl[i] + (rest > 0 ? 1 : 0);
                } else {
                    v[i] = a.fixed_splits > 0 ? max(1, min(a.fixed_splits, tiles))
                                              : max(1, (int)((uint32_t)(tiles + tpi - 1) / (uint32_t)tpi));
                    fl[i] = v[i];
                }
                S.ns[b] = v[i];
            }
            sp[i] = v[i] > 1 ? 1 : 0;
            run += v[i];
            nsp += sp[i];
            nfl += fl[i];
        }
        int incl = run, incl_sp = nsp, incl_fl = nfl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            const int y = __shfl_up_sync(0xffffffffu, incl_sp, o);
            const int z = __shfl_up_sync(0xffffffffu, incl_fl, o);
            if (lane >= o) { incl += x; incl_sp += y; incl_fl += z; }
        }
        const int first = __shfl_sync(0xffffffffu, incl_fl, 31);    // items before the remainders
        int acc = incl - run, acc_sp = incl_sp - nsp, acc_fl = incl_fl - nfl;
        int acc_re = acc - acc_fl;                                  // remainders before this rank
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int k = lane * K + i;
            if (k < B) {
                const int b = S.by_rank[k];
                S.base[b] = acc;
                if (sp[i]) S.split[acc_sp] = b;
                int part = -1;                                      // this item's part of sequence b
                if (item >= acc_fl && item < acc_fl + fl[i]) part = item - acc_fl;
                if (v[i] > fl[i] && item == first + acc_re) part = fl[i];
                if (part >= 0) {
                    const int parts = v[i] > fl[i] ? 0 : v[i];      // equal ones, or chunks and a remainder
                    const int per = parts > 0 ? (int)((uint32_t)(S.tb[b] + parts - 1) / (uint32_t)parts) : chunk;
                    S.item.b = b;
                    S.item.tile_begin = part * per;
                    S.item.tile_end = min(S.tb[b], (part + 1) * per);
                    S.item.part = v[i] > 1 ? acc + part : -1;
                    S.item_len = S.len[b];
                }
                acc += v[i];
                acc_fl += fl[i];
                acc_re += v[i] - fl[i];
            }
            acc_sp += sp[i];
        }
        if (lane == 31) {
            S.n_items = incl;
            S.n_split = incl_sp;
        }
    }
    __syncthreads();
}

}  // namespace dec
}  // namespace qkmla
