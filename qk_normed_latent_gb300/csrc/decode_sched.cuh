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
    int base[kMaxBSched];      // first item of sequence b
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
template <bool SPLITS_ONLY = false>
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
    const int tpi = max(max((float)m <= 1.25f * ideal ? m : (int)ceilf(ideal), a.min_tokens / a.tile), 1);
    if constexpr (SPLITS_ONLY) {
        if (a.fixed_splits == 0 && m <= tpi) {      // uniform
            if (tid == 0) S.n_split = 0;
            __syncthreads();
            return;
        }
    }
    for (int b = warp; b < B; b += nw) {
        const int mine = S.tb[b];
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
        int v[K], sp[K];
        int run = 0, nsp = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int k = lane * K + i;
            v[i] = 0;
            if (k < B) {
                const int b = S.by_rank[k], tiles = S.tb[b];
                v[i] = a.fixed_splits > 0 ? max(1, min(a.fixed_splits, tiles))
                                          : max(1, (int)((uint32_t)(tiles + tpi - 1) / (uint32_t)tpi));
                S.ns[b] = v[i];
            }
            sp[i] = v[i] > 1 ? 1 : 0;
            run += v[i];
            nsp += sp[i];
        }
        int incl = run, incl_sp = nsp;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            const int y = __shfl_up_sync(0xffffffffu, incl_sp, o);
            if (lane >= o) { incl += x; incl_sp += y; }
        }
        int acc = incl - run, acc_sp = incl_sp - nsp;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int k = lane * K + i;
            if (k < B) {
                const int b = S.by_rank[k];
                S.base[b] = acc;
                if (sp[i]) S.split[acc_sp] = b;
                if (item >= acc && item < acc + v[i]) {
                    const int per = (int)((uint32_t)(S.tb[b] + v[i] - 1) / (uint32_t)v[i]);
                    S.item.b = b;
                    S.item.tile_begin = (item - acc) * per;
                    S.item.tile_end = min(S.tb[b], (item - acc + 1) * per);
                    S.item.part = v[i] > 1 ? item : -1;
                    S.item_len = S.len[b];
                }
                acc += v[i];
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
