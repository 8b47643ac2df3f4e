// qkmla_prefill: attention of query tiles over the recovered keys and values, and the join of cut rows.
//
// A query tile is 256 rows, tokens x the heads of one unit (heads that share a key and a value matrix), in
// two halves of 128.  Keys and values of a token tile serve all 256, so that a unit of 16 heads reads a key
// once for 16 query tokens, and a causal edge is at most one tile wide.
//
//   S = Q K^T            M = 128 rows, N = 128 tokens, K = d_h + d_r, into TMEM (a half's 128 columns)
//   softmax              thread = row: reads S, moves its running maximum, writes P (fp16) over S
//   O += P V             M = 128, N = d_v, K = 128 tokens, A = P out of TMEM, O in TMEM (128 columns a half)
//
// Warps 0-3 and 4-7 are the two halves' softmax, warp 8 loads (bulk copies of prepared blocks into a ring),
// warp 9 issues (10 and 11 make the warpgroup whole).  The halves alternate: while one half's S is worked on, the other's PV and the next QK run:
// PV0(j) QK0(j+1) PV1(j) QK1(j+1).  The products of one thread run in order, so QK may write S over the P
// that the PV ahead of it reads, and a half whose S(j) is complete knows that its PV(j-1) is.
//
// Numbers.  S is in units of the row's factor c (softmax_scale, log2 e and the query's power of two).  The
// tile's values are 2^-E of themselves, so a row's weights are P_t = 2^(c S_t + E + 7 - m) with m a running
// maximum of c S_t + E, moved only when it is exceeded by 2^8: P <= 2^15 fits fp16, whose normal range then
// reaches 2^-21 below the largest weight.  The sum of the softmax is kept in fp32 from the unrounded
// weights, 2^-E of each tile's; O, in TMEM, is in fp32.  fp16 instead of bf16 because keys and queries are
// normalised (bounded) and a tile's values have an exponent of their own: 8 times smaller roundings at the
// same rate.  A tile whose latents differ too much holds its values as bf16, and its P is bf16 too.
//
// Work.  A CTA an SM takes an even share of the list of (unit, query tile, token tile); a query tile that is
// cut leaves its parts in the workspace and prefill_join_kernel adds them, by weights 2^(m_s - max m).
//
// Bound: the tensor core (20 products of 128 x 128 x 16 a half and token tile for d_h + d_r + d_v = 320,
// 1300 cycles), next to it shared-memory bandwidth (each product reads 4 KB of B and, for QK, 4 KB of A).
#include "prefill.cuh"

namespace qkmla {
namespace pf {
namespace {

using namespace tc;

constexpr int kThreadsA = 384;
// Registers: 384 threads start with 168 each, the most that 65536 allow.  The softmax keeps a row of 128 logits,
// so the warpgroup of the loads and products gives up 96 of its 168 and each half's takes 48 of them:
// 2 x 216 + 72 = 3 x 168.
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * 168, "register split");
constexpr int kUnits = 8;                  // ring, in blocks
constexpr int kGroups = 8;                 // barriers of groups (a token tile's key blocks, or its value blocks)

struct __align__(8) Shared {
    uint64_t full[kGroups], empty[kGroups];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t done;
    uint32_t tmem;
    int fail;
    int issued;                            // groups whose copies were issued
    int q_issued;                          // query tiles whose copies were issued
};

template <int DH>
constexpr int smem_bytes() { return (2 * (DH / 64 + 1) + kUnits) * kBlock + 1024 + 1024; }

// One CTA's part of the list, walked alike by every warp.
struct Walk {
    Place at, end;
    int64_t one;
    bool first;

    // The next piece: tiles [t0, t1) of slot j of unit u, of nt; false at the end.
    struct Piece {
        int u, j, t0, t1, nt;
        int4 a, b;                         // qinfo
    };
    __device__ __forceinline__ bool next(const Params& p, Piece& s) {
        for (;;) {
            if (at.u > end.u || (at.u == end.u && at.j > end.j) || at.u >= p.units) return false;
            const bool last = at.u == end.u && at.j == end.j;
            if (last && end.t == 0) return false;
            s.u = at.u;
            s.j = at.j;
            s.t0 = first ? at.t : 0;
            first = false;
            if (++at.j == p.nq) { at.j = 0; ++at.u; }
            s.a = p.qinfo[2 * s.j];
            if (s.a.x < 0) continue;                       // an unused slot
            s.b = p.qinfo[2 * s.j + 1];
            s.nt = s.a.z;
            s.t1 = last ? end.t : s.nt;
            if (s.t0 == s.t1 && s.nt > 0) continue;
            return true;
        }
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Named barriers cannot be used where a thread may have given up; every wait below ends by itself.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, Shared* sh, int* status) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = dec::globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (*(volatile int*)&sh->fail) return false;
            if (dec::globaltimer() - t0 > dec::kWaitNs) {
                report(status, QKMLA_ERR_TIMEOUT);
                *(volatile int*)&sh->fail = 1;
                return false;
            }
        }
    }
}

template <int DH, int DV, typename OT>
__global__ void __launch_bounds__(kThreadsA, 1) prefill_attend_kernel(const __grid_constant__ Params p) {
    constexpr int KU = DH / 64 + 1;                        // blocks of a key tile
    constexpr int VU = DV / 64;
    constexpr int kHalf = KU * kBlock;                     // a half's queries
    constexpr uint32_t kS = 0, kO = 256;                   // TMEM: S of half h at 128 h, O at 256 + 128 h
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint8_t* ring = sm + 2 * kHalf;
    Shared* sh = reinterpret_cast<Shared*>(ring + kUnits * kBlock);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kGroups; ++i) { mbar_init(&sh->full[i], 1); mbar_init(&sh->empty[i], 1); }
        mbar_init(&sh->q_full, 1);
        mbar_init(&sh->q_empty, 1);
        for (int i = 0; i < 2; ++i) { mbar_init(&sh->s_full[i], 1); mbar_init(&sh->p_full[i], 128); mbar_init(&sh->o_full[i], 1); }
        mbar_init(&sh->done, 1);
        sh->fail = 0;
        sh->issued = 0;
        sh->q_issued = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&sh->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    pdl_wait();
    pdl_trigger();

    Walk walk;
    walk.one = p.pre[p.nq];
    const int64_t all = walk.one * p.units;
    const int n_cta = sharing(p, all);
    const int cta = blockIdx.x;
    const bool busy = all > 0 && cta < n_cta;              // uniform
    if (busy) {
        walk.at = place_of(p, share_start(all, n_cta, cta), walk.one);
        walk.end = place_of(p, share_start(all, n_cta, cta + 1), walk.one);
        walk.first = true;
    }

    if (!busy) {
    } else if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
      if (warp == 8) {
        // ---- loads ----
        if (lane == 0) {
            int group = 0, unit = 0;                       // issued so far
            int freed = 0, freed_units = 0;
            int tiles_q = 0;
            bool ok = true;
            auto put = [&](const uint8_t* a, int na, const uint8_t* b2, int nb) {      // a group: na blocks at a, nb at b2
                const int n = na + nb;
                while (ok && unit + n - kUnits > freed_units) {
                    ok = wait_or_fail(&sh->empty[freed % kGroups], (freed / kGroups) & 1, sh, p.status);
                    freed_units += (freed & 1) ? VU : KU;
                    ++freed;
                }
                if (!ok) return;
                uint64_t* bar = &sh->full[group % kGroups];
                mbar_arrive_expect_tx(bar, n * kBlock);
                for (int i = 0; i < n; ++i) {
                    bulk_load(ring + (unit % kUnits) * kBlock, i < na ? a + (size_t)i * kBlock : b2 + (size_t)(i - na) * kBlock, kBlock, bar);
                    ++unit;
                }
                ++group;
                *(volatile int*)&sh->issued = group;
            };
            typename Walk::Piece s;
            while (ok && walk.next(p, s)) {
                if (s.t0 == s.t1) continue;
                const int4 seq = p.seq[s.a.x];
                const int g = (int)((int64_t)s.u * p.G / p.units), gv = (int)((int64_t)s.u * p.Gv / p.units);
                const bool two = s.b.z * p.hp > 128;
                for (int t = s.t0; t < s.t1 && ok; ++t) {
                    const size_t tile = (size_t)seq.y + (t < s.a.w ? t : t + s.b.x);
                    put(p.kc + (tile * p.G + g) * (size_t)((KU - 1) * kBlock), KU - 1, p.krope + tile * kBlock, 1);
                    if (t == s.t0 && ok) {
                        // the queries, once the last tile's are no longer read
                        if (tiles_q > 0) ok = wait_or_fail(&sh->q_empty, (tiles_q - 1) & 1, sh, p.status);
                        if (!ok) break;
                        const int bytes = (two ? 2 : 1) * kHalf;
                        mbar_arrive_expect_tx(&sh->q_full, bytes);
                        const uint8_t* q = p.qt + ((size_t)s.u * p.nq + s.j) * (size_t)(2 * kHalf);
                        for (int i = 0; i < (two ? 2 : 1); ++i) bulk_load(sm + i * kHalf, q + (size_t)i * kHalf, kHalf, &sh->q_full);
                        ++tiles_q;
                        *(volatile int*)&sh->q_issued = tiles_q;
                    }
                    put(p.v + (tile * p.Gv + gv) * (size_t)(VU * kBlock), VU, nullptr, 0);
                }
            }
        }
        __syncwarp();
      } else if (warp == 9) {
        // ---- products ----
        constexpr uint32_t bf = (1u << 7) | (1u << 10);
        const uint32_t id_s = idesc_bf16(128, 128, 0, 0) & ~bf;
        const uint32_t id_o = idesc_bf16(128, DV, 0, 1) & ~bf;
        const uint32_t id_o64 = idesc_bf16(128, 64, 0, 1) & ~bf;
        const int rope_steps = p.d_r / 16;
        int group = 0, unit = 0, tiles_q = 0;
        uint32_t p_phase[2] = {0, 0};
        bool ok = true;
        auto block_at = [&](int u) { return smem_u32(ring + (u % kUnits) * kBlock); };
        // S of half h from the key blocks at `u`
        auto qk = [&](int h, int u) {
            const uint32_t q = smem_u32(sm + h * kHalf);
            if (elect_one()) {
#pragma unroll
                for (int blk = 0; blk < KU - 1; ++blk) {
                    const uint32_t k = block_at(u + blk);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16(tmem + kS + h * 128, smem_desc(q + blk * kBlock + kk * 32, 16, 1024, kSwizzle128B),
                                 smem_desc(k + kk * 32, 16, 1024, kSwizzle128B), id_s, (blk > 0 || kk > 0) ? 1u : 0u);
                }
                const uint32_t k = block_at(u + KU - 1);
                for (int kk = 0; kk < rope_steps; ++kk)
                    mma_bf16(tmem + kS + h * 128, smem_desc(q + (KU - 1) * kBlock + kk * 32, 16, 1024, kSwizzle128B),
                             smem_desc(k + kk * 32, 16, 1024, kSwizzle128B), id_s, 1u);
                mma_commit(&sh->s_full[h]);
            }
            __syncwarp();
        };
        auto pv = [&](int h, int u, bool as_bf, bool acc) {
            const uint32_t v0 = block_at(u), v1 = block_at(u + VU - 1);
            const uint32_t fmt = as_bf ? bf : 0u;
            if (elect_one()) {
                if (VU == 1 || v1 > v0) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16_tmem_a(tmem + kO + h * 128, tmem + kS + h * 128 + kk * 8, smem_desc(v0 + kk * 2048, kBlock, 1024, kSwizzle128B),
                                        id_o | fmt, (acc || kk > 0) ? 1u : 0u);
                } else {
                    // the value blocks wrap around the ring's end: 64 columns at a time
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        mma_bf16_tmem_a(tmem + kO + h * 128, tmem + kS + h * 128 + kk * 8, smem_desc(v0 + kk * 2048, kBlock, 1024, kSwizzle128B),
                                        id_o64 | fmt, (acc || kk > 0) ? 1u : 0u);
                        mma_bf16_tmem_a(tmem + kO + h * 128 + 64, tmem + kS + h * 128 + kk * 8, smem_desc(v1 + kk * 2048, kBlock, 1024, kSwizzle128B),
                                        id_o64 | fmt, (acc || kk > 0) ? 1u : 0u);
                    }
                }
            }
            __syncwarp();
        };
        auto wait_group = [&](int g) { return wait_or_fail(&sh->full[g % kGroups], (g / kGroups) & 1, sh, p.status); };
        auto commit = [&](uint64_t* bar) {
            if (elect_one()) mma_commit(bar);
            __syncwarp();
        };
        typename Walk::Piece s;
        while (ok && walk.next(p, s)) {
            if (s.t0 == s.t1) continue;
            const int4 seq = p.seq[s.a.x];
            const int halves = s.b.z * p.hp > 128 ? 2 : 1;
            const int n = s.t1 - s.t0;
            auto tile_of = [&](int t) { return seq.y + (t < s.a.w ? t : t + s.b.x); };
            int info = p.tinfo[tile_of(s.t0)];
            if (!(ok = wait_group(group))) break;
            if (!(ok = wait_or_fail(&sh->q_full, tiles_q & 1, sh, p.status))) break;
            ++tiles_q;
            tc_fence_after();
            for (int h = 0; h < halves; ++h) qk(h, unit);
            commit(&sh->empty[group % kGroups]);
            if (n == 1) commit(&sh->q_empty);
            ++group;
            unit += KU;
            for (int j = 0; j < n && ok; ++j) {
                const int vu = unit, ku = unit + VU, gv = group, gk = group + 1;
                const bool as_bf = (info & 256) != 0, more = j + 1 < n;
                if (more) info = p.tinfo[tile_of(s.t0 + j + 1)];
                for (int h = 0; h < halves; ++h) {
                    ok = wait_or_fail(&sh->p_full[h], p_phase[h], sh, p.status);
                    if (!ok) break;
                    p_phase[h] ^= 1;
                    if (h == 0 && !(ok = wait_group(gv))) break;
                    tc_fence_after();
                    pv(h, vu, as_bf, j > 0);
                    if (h == halves - 1) commit(&sh->empty[gv % kGroups]);
                    if (!more) {
                        commit(&sh->o_full[h]);
                    } else {
                        if (h == 0 && !(ok = wait_group(gk))) break;
                        tc_fence_after();
                        qk(h, ku);
                        if (h == halves - 1) commit(&sh->empty[gk % kGroups]);
                    }
                }
                if (more && j + 2 == n && ok) commit(&sh->q_empty);
                group += more ? 2 : 1;
                unit += VU + (more ? KU : 0);
            }
        }
        commit(&sh->done);
      }
    } else {
        // ---- softmax: thread = row ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int h = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t t_s = tmem + lane_base + kS + h * 128, t_o = tmem + lane_base + kO + h * 128;
        const int* we = reinterpret_cast<const int*>(p.weights);
        uint32_t s_phase = 0, o_phase = 0;
        bool ok = true;
        typename Walk::Piece s;
        while (walk.next(p, s)) {
            if (h == 1 && s.b.z * p.hp <= 128) continue;
            const int4 seq = p.seq[s.a.x];
            const int rt = h * 128 + row, i = rt / p.hp;               // the row's query within the tile
            const bool there = i < s.b.z;
            const int n_row = there ? s.b.y + i : 0;                    // causal length
            const int n_hi = s.b.y + s.b.z - 1;
            const float c = p.qc[((size_t)s.u * p.nq + s.j) * kRowsQ + rt];
            float m = -INFINITY, sum = 0.f;
            auto tile_at = [&](int t) { return t < s.a.w ? t : t + s.b.x; };
            int info = s.t0 < s.t1 ? p.tinfo[seq.y + tile_at(s.t0)] : 0;
            for (int t = s.t0; t < s.t1 && ok; ++t) {
                const int first = tile_at(t) * kTile;
                const int e = (info & 255) - 64;
                const bool as_bf = (info & 256) != 0;
                if (t + 1 < s.t1) info = p.tinfo[seq.y + tile_at(t + 1)];
                ok = wait_or_fail(&sh->s_full[h], s_phase, sh, p.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                s_phase ^= 1;
                tc_fence_after();
                float x[128];
                tmem_ld64(t_s, *reinterpret_cast<uint32_t(*)[64]>(x));
                tmem_ld64(t_s + 64, *reinterpret_cast<uint32_t(*)[64]>(x + 64));
                tmem_wait_ld();
                // tiles that some row does not see whole (uniform over the tile's rows)
                const bool edge = first + kTile > s.b.y || (p.window > 0 && first < n_hi - p.window && first + kTile > p.sinks);
                if (edge) {
                    const int end = n_row - first;
                    const int from = p.window > 0 ? n_row - p.window - first : -1, sink = p.window > 0 ? p.sinks - first : -1;
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k >= end || (k < from && k >= sink)) x[k] = -INFINITY;
                }
                float top[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
                for (int k = 4; k < 128; k += 4) {
                    top[0] = fmaxf(top[0], fmaxf(x[k], x[k + 2]));
                    top[1] = fmaxf(top[1], fmaxf(x[k + 1], x[k + 3]));
                }
                const float cand = fmaf(fmaxf(top[0], top[1]), c, (float)e);
                const bool move = cand > m + 8.f;
                if (__any_sync(0xffffffffu, move)) {
                    const float m2 = move ? cand : m;
                    const float a = move ? ex2(m - m2) : 1.f;           // 0 while nothing was seen
                    sum *= a;
                    if (t > s.t0) {
#pragma unroll
                        for (int k = 0; k < DV; k += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + k, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * a);
                            tmem_st16(t_o + k, o);
                        }
                    }
                    m = m2;
                }
                const float off = (float)(e + 7) - (m == -INFINITY ? 0.f : m);
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 128; k += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        x[k + q] = ex2(fmaf(x[k + q], c, off));
                        part[q & 3] += x[k + q];
                    }
                    if (as_bf) {
#pragma unroll
                        for (int q = 0; q < 16; ++q) w[q] = pack_bf16(x[k + 2 * q], x[k + 2 * q + 1]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 16; ++q) w[q] = pack_f16(x[k + 2 * q], x[k + 2 * q + 1]);
                    }
                    tmem_st16(t_s + k / 2, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sh->p_full[h]);
                sum = fmaf((part[0] + part[1]) + (part[2] + part[3]), pow2i(-e), sum);
            }
            if (s.t0 < s.t1 && ok) ok = wait_or_fail(&sh->o_full[h], o_phase, sh, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            if (s.t0 < s.t1) {
                o_phase ^= 1;
                tc_fence_after();
            }
            const int gv = (int)((int64_t)s.u * p.Gv / p.units);
            if (whole) {
                const float inv = sum == 0.f ? 0.f : ldexpf(1.f / sum, we[p.G + gv]);
                const int head = s.u * p.hp + rt % p.hp;
                const int64_t r = seq.z + s.a.y + i;
                OT* dst = reinterpret_cast<OT*>(p.o) + (r * p.H + head) * DV;
#pragma unroll 1
                for (int k = 0; k < DV; k += 32) {
                    float o[32];
                    if (s.t0 < s.t1) {
                        tmem_ld16(t_o + k, *reinterpret_cast<uint32_t(*)[16]>(o));
                        tmem_ld16(t_o + k + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int q = 0; q < 32; ++q) o[q] = sum == 0.f ? 0.f : o[q] * inv;
                    if (there) {
                        if constexpr (sizeof(OT) == 4) {
#pragma unroll
                            for (int q = 0; q < 8; ++q) reinterpret_cast<float4*>(dst + k)[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                        } else {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                reinterpret_cast<uint4*>(dst + k)[q] = make_uint4(pack_bf16(o[8 * q], o[8 * q + 1]), pack_bf16(o[8 * q + 2], o[8 * q + 3]),
                                                                                  pack_bf16(o[8 * q + 4], o[8 * q + 5]), pack_bf16(o[8 * q + 6], o[8 * q + 7]));
                        }
                    }
                }
                if (there && p.lse) p.lse[r * p.H + head] = sum == 0.f ? -INFINITY : (m - 7.f) * kLn2 + logf(sum);
            } else {
                const size_t part = (size_t)(2 * cta + (s.t0 > 0 ? 0 : 1)) * kRowsQ + rt;
                float* dst = p.part_o + part * DV;
#pragma unroll 1
                for (int k = 0; k < DV; k += 32) {
                    float o[32];
                    tmem_ld16(t_o + k, *reinterpret_cast<uint32_t(*)[16]>(o));
                    tmem_ld16(t_o + k + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
                    tmem_wait_ld();
                    if (there) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) reinterpret_cast<float4*>(dst + k)[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    }
                }
                if (there) p.part_ml[part] = make_float2(m, sum);
            }
            tc_fence_before();                                          // the next tile's PV writes O after this half's P
        }
    }
    __syncthreads();
    if (busy) {
        // a CTA that gave up waits for its copies in flight, and always for its products
        wait_or_fail(&sh->done, 0, sh, p.status);
        if (*(volatile int*)&sh->fail && tid == 0) {
            dec::wait_bounded(&sh->done, 0, p.status);
            const int n = *(volatile int*)&sh->issued, q = *(volatile int*)&sh->q_issued;
            for (int g = max(0, n - kGroups); g < n; ++g) dec::wait_bounded(&sh->full[g % kGroups], (g / kGroups) & 1, p.status);
            if (q > 0) dec::wait_bounded(&sh->q_full, (q - 1) & 1, p.status);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// join of cut query tiles
// ---------------------------------------------------------------------------
// Block (k, y): rows 16 y .. 16 y + 15 of the query tile that the boundary between CTA k and k + 1 cuts, if no
// earlier boundary cuts it.  Half a warp a row of 64, a warp a row of 128 values.
constexpr int kThreadsJ = 128;
constexpr int kRowsJ = 16;

template <int DV, typename OT>
__global__ void __launch_bounds__(kThreadsJ) prefill_join_kernel(const __grid_constant__ Params p) {
    pdl_wait();
    pdl_trigger();
    const int64_t one = p.pre[p.nq], all = one * p.units;
    const int n_cta = sharing(p, all);
    const int k = blockIdx.x + 1;
    if (all == 0 || k >= n_cta) return;
    const Place at = place_of(p, share_start(all, n_cta, k), one);
    if (!at.inside()) return;
    if (k > 1) {
        const Place prev = place_of(p, share_start(all, n_cta, k - 1), one);
        if (prev.inside() && prev.u == at.u && prev.j == at.j) return;
    }
    // parts: CTA k - 1's last piece, then the first pieces of CTAs k .. last - 1 (one that got no tile has none)
    __shared__ int parts[160];
    __shared__ int count;
    if (threadIdx.x < 32) {
        int n = 0;
        if (threadIdx.x == 0) parts[0] = 2 * (k - 1) + 1;
        n = 1;
        Place from = at;
        for (int q = k; q < n_cta; ++q) {
            const Place to = place_of(p, share_start(all, n_cta, q + 1), one);
            const bool same = to.u == at.u && to.j == at.j && to.t < at.nt;
            if (!(same && to.t == from.t)) {
                if (threadIdx.x == 0) parts[n] = 2 * q;
                ++n;
            }
            if (!same) break;
            from = to;
        }
        if (threadIdx.x == 0) count = n;
    }
    __syncthreads();
    const int n = count;
    const int4 a = p.qinfo[2 * at.j], b = p.qinfo[2 * at.j + 1];
    const int4 seq = p.seq[a.x];
    const int gv = (int)((int64_t)at.u * p.Gv / p.units);
    const int e = reinterpret_cast<const int*>(p.weights)[p.G + gv];
    constexpr int kLanes = DV / 4;                          // lanes a row, 4 values each
    constexpr int kPerPass = kThreadsJ / kLanes;
    for (int q = threadIdx.x / kLanes; q < kRowsJ; q += kPerPass) {
        const int rt = blockIdx.y * kRowsJ + q, i = rt / p.hp;
        if (i >= b.z) continue;
        float top = -INFINITY;
        for (int s = 0; s < n; ++s) top = fmaxf(top, p.part_ml[(size_t)parts[s] * kRowsQ + rt].x);
        float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        const int col = threadIdx.x % kLanes * 4;
        for (int s = 0; s < n; ++s) {
            const size_t row = (size_t)parts[s] * kRowsQ + rt;
            const float2 ml = p.part_ml[row];
            // a part that saw nothing has m = -inf and weight 0, unless its sum is NaN (a key that is not finite)
            const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - top);
            if (w == 0.f && ml.y == ml.y) continue;
            const float4 v = *reinterpret_cast<const float4*>(p.part_o + row * DV + col);
            sum = fmaf(w, ml.y, sum);
            o[0] = fmaf(w, v.x, o[0]); o[1] = fmaf(w, v.y, o[1]); o[2] = fmaf(w, v.z, o[2]); o[3] = fmaf(w, v.w, o[3]);
        }
        const int head = at.u * p.hp + rt % p.hp;
        const int64_t r = seq.z + a.y + i;
        const float inv = sum == 0.f ? 0.f : ldexpf(1.f / sum, e);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = sum == 0.f ? 0.f : o[c] * inv;
        OT* dst = reinterpret_cast<OT*>(p.o) + (r * p.H + head) * DV + col;
        if constexpr (sizeof(OT) == 4) *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
        else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
        if (col == 0 && p.lse) p.lse[r * p.H + head] = sum == 0.f ? -INFINITY : (top - 7.f) * kLn2 + logf(sum);
    }
}

template <int DH, int DV, typename OT>
int launch(const Params& p, cudaStream_t s) {
    auto k = prefill_attend_kernel<DH, DV, OT>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<DH>()) != cudaSuccess) return QKMLA_ERR_CUDA;
    if (launch_pdl(k, dim3(p.ctas), dim3(kThreadsA), smem_bytes<DH>(), s, p) != cudaSuccess) return QKMLA_ERR_CUDA;
    if (p.ctas < 2) return QKMLA_OK;
    return launch_pdl(prefill_join_kernel<DV, OT>, dim3(p.ctas - 1, kRowsQ / kRowsJ), dim3(kThreadsJ), 0, s, p) == cudaSuccess ? QKMLA_OK
                                                                                                                             : QKMLA_ERR_CUDA;
}

template <typename OT>
int launch_dims(const Params& p, cudaStream_t s) {
    if (p.d_h == 128) return p.d_v == 128 ? launch<128, 128, OT>(p, s) : launch<128, 64, OT>(p, s);
    return p.d_v == 128 ? launch<64, 128, OT>(p, s) : launch<64, 64, OT>(p, s);
}

}  // namespace

int launch_attend(const Params& p, int o_dtype, cudaStream_t s) {
    return o_dtype == QKMLA_F32 ? launch_dims<float>(p, s) : launch_dims<__nv_bfloat16>(p, s);
}

}  // namespace pf
}  // namespace qkmla

using namespace qkmla;

namespace {

// Argument checks and everything that follows from the sizes; pointers into the workspace at `base`.
int make_params(const qkmla_prefill_args* a, bool sizes_only, pf::Params* p, size_t* bytes) {
    if (!a) return QKMLA_ERR_INVALID;
    if (a->B < 1 || a->rows < 0 || a->H < 1 || a->G < 1 || a->G_v < 1 || a->d_c < 1 || a->d_h < 1 || a->d_r < 1 || a->d_v < 1)
        return QKMLA_ERR_INVALID;
    if (a->H % a->G || a->H % a->G_v) return QKMLA_ERR_INVALID;
    if (a->page_size < 1 || a->max_pages < 1 || a->num_slots < 1 || a->num_slots % a->page_size) return QKMLA_ERR_INVALID;
    if ((int64_t)a->max_pages * a->page_size > INT32_MAX - 4096) return QKMLA_ERR_INVALID;
    if (a->total_tokens < 0 || a->window < 0 || a->sinks < 0 || (a->sinks > 0 && a->window == 0)) return QKMLA_ERR_INVALID;
    if (!(a->softmax_scale > 0.f) || !(a->eps >= 0.f)) return QKMLA_ERR_INVALID;
    const bool q8 = a->cache_dtype == QKMLA_E4M3;
    if (a->flags & QKMLA_FLAG_PLAIN_MLA) return QKMLA_ERR_UNSUPPORTED;
    if (!q8 && a->cache_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    if (a->q_dtype != QKMLA_F32 && a->q_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    if (a->o_dtype != QKMLA_F32 && a->o_dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    const int units = a->G > a->G_v ? a->G : a->G_v, hp = a->H / units;
    if (units % a->G || units % a->G_v || hp > 128 || (hp & (hp - 1))) return QKMLA_ERR_UNSUPPORTED;
    if ((a->d_h != 64 && a->d_h != 128) || (a->d_v != 64 && a->d_v != 128) || (a->d_r != 32 && a->d_r != 64)) return QKMLA_ERR_UNSUPPORTED;
    if (a->d_c % 64 || a->d_c > 512 || a->B > 4096 || units > 512) return QKMLA_ERR_UNSUPPORTED;
    if ((int64_t)a->rows * a->H > INT32_MAX || a->total_tokens / pf::kTile + a->B > (1 << 24)) return QKMLA_ERR_UNSUPPORTED;
    *p = pf::Params{};
    p->page_size = a->page_size;
    p->max_pages = a->max_pages;
    p->num_pages = a->num_slots / a->page_size;
    p->B = a->B;
    p->rows = a->rows;
    p->H = a->H;
    p->G = a->G;
    p->Gv = a->G_v;
    p->d_c = a->d_c;
    p->d_h = a->d_h;
    p->d_r = a->d_r;
    p->d_v = a->d_v;
    p->scale_log2 = a->softmax_scale * kLog2e;
    p->eps = a->eps;
    const int64_t longest = (int64_t)a->max_pages * a->page_size;
    p->window = (int)(a->window < longest ? a->window : a->window ? longest : 0);
    p->sinks = (int)(a->sinks < longest ? a->sinks : longest);
    p->ak_f16 = (a->flags & QKMLA_FLAG_ALPHA_F16) ? 1 : 0;
    p->total_tokens = a->total_tokens;
    p->units = units;
    p->hp = hp;
    p->tq = pf::kRowsQ / hp;
    p->nq = a->rows / p->tq + a->B;
    p->max_tiles = (int)(a->total_tokens / pf::kTile) + a->B;
    p->ctas = device_sm_count();
    if (p->ctas <= 0) return QKMLA_ERR_CUDA;
    if (p->ctas > 158) p->ctas = 158;                      // the join's list of parts
    uintptr_t at = (uintptr_t)a->workspace;
    auto take = [&](size_t n) {
        const uintptr_t r = at;
        at += (n + 255) & ~(size_t)255;
        return r;
    };
    const size_t tiles = p->max_tiles, nq = p->nq;
    p->seq = (int4*)take(sizeof(int4) * a->B);
    p->qinfo = (int4*)take(sizeof(int4) * 2 * nq);
    p->pre = (int64_t*)take(8 * (nq + 1));
    p->tinfo = (int*)take(4 * tiles);
    p->part_ml = (float2*)take(sizeof(float2) * 2 * p->ctas * pf::kRowsQ);
    p->qc = (float*)take(4 * (size_t)units * nq * pf::kRowsQ);
    p->part_o = (float*)take(4 * (size_t)2 * p->ctas * pf::kRowsQ * a->d_v);
    p->krope = (uint8_t*)take(tiles * pf::kBlock);
    p->kc = (uint8_t*)take(tiles * a->G * (a->d_h / 64) * pf::kBlock);
    p->v = (uint8_t*)take(tiles * a->G_v * (a->d_v / 64) * pf::kBlock);
    p->qt = (uint8_t*)take((size_t)units * nq * 2 * (a->d_h / 64 + 1) * pf::kBlock);
    *bytes = at - (uintptr_t)a->workspace;
    if (sizes_only) return QKMLA_OK;
    if (q8 != (a->kv_scale != nullptr)) return QKMLA_ERR_INVALID;
    for (int64_t st : {a->q_row_stride, a->q_head_stride, a->qr_row_stride, a->qr_head_stride})
        if (st % 4) return QKMLA_ERR_INVALID;
    if (a->rows == 0) return QKMLA_OK;
    if (!a->q || !a->q_rope || !a->gamma_q || !a->gamma_k || !a->weights || !a->kv_cache || !a->ak_cache || !a->chunk_start ||
        !a->seq_lens || !a->o)
        return QKMLA_ERR_INVALID;
    for (const void* ptr : {a->q, a->q_rope, a->weights, a->kv_cache, (const void*)a->o})
        if ((uintptr_t)ptr % 16) return QKMLA_ERR_INVALID;
    for (const void* ptr : {(const void*)a->gamma_q, (const void*)a->gamma_k, (const void*)a->gamma_rope_q, (const void*)a->kv_scale,
                            (const void*)a->chunk_start, (const void*)a->seq_lens, (const void*)a->page_table, (const void*)a->lse})
        if ((uintptr_t)ptr % 4) return QKMLA_ERR_INVALID;
    if ((uintptr_t)a->ak_cache % (p->ak_f16 ? 2 : 4)) return QKMLA_ERR_INVALID;
    if (!a->workspace || a->workspace_bytes < *bytes) return QKMLA_ERR_WORKSPACE;
    if ((uintptr_t)a->workspace % 256) return QKMLA_ERR_INVALID;
    p->q = a->q;
    p->q_rope = a->q_rope;
    p->q_row = a->q_row_stride;
    p->q_head = a->q_head_stride;
    p->qr_row = a->qr_row_stride;
    p->qr_head = a->qr_head_stride;
    p->gamma_q = a->gamma_q;
    p->gamma_k = a->gamma_k;
    p->gamma_rope = a->gamma_rope_q;
    p->weights = (const uint8_t*)a->weights;
    p->kv = (const uint8_t*)a->kv_cache;
    p->kv_scale = a->kv_scale;
    p->ak = a->ak_cache;
    p->chunk_start = a->chunk_start;
    p->seq_lens = a->seq_lens;
    p->page_table = a->page_table;
    p->o = a->o;
    p->lse = a->lse;
    p->status = device_status_ptr();
    return QKMLA_OK;
}

}  // namespace

extern "C" size_t qkmla_prefill_workspace_size(const qkmla_prefill_args* a) {
    pf::Params p;
    size_t bytes = 0;
    return make_params(a, true, &p, &bytes) == QKMLA_OK ? bytes : 0;
}

extern "C" int qkmla_prefill(const qkmla_prefill_args* a, void* stream) {
    pf::Params p;
    size_t bytes = 0;
    int rc = make_params(a, false, &p, &bytes);
    if (rc != QKMLA_OK || a->rows == 0) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if ((rc = pf::launch_query(p, a->q_dtype == QKMLA_BF16, s)) != QKMLA_OK) return rc;
    if ((rc = pf::launch_expand(p, a->cache_dtype == QKMLA_E4M3, s)) != QKMLA_OK) return rc;
    return pf::launch_attend(p, a->o_dtype, s);
}
