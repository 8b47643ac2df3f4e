// qkmla_prefill: attention of query tiles over the recovered keys and values, and the join of cut rows.
//
// A query tile is 256 rows, tokens x the heads of one unit (heads that share a key and a value matrix), in
// two halves of 128.  Keys and values of a token tile serve all 256, so that a unit of 16 heads reads a key
// once for 16 query tokens, and a causal edge is at most one tile wide.
//
//   S = Q K^T            M = 128 rows, N = 128 tokens, K = d_h + d_r, into TMEM (a half's 128 columns)
//   softmax              thread = row: holds S in registers (its maximum comes with the TMEM load), moves its
//                        running maximum, writes P over S; the product waits for 64 tokens at a time
//   O += P V             M = 128, N = d_v, K = 128 tokens, A = P out of TMEM, O in TMEM (128 columns a half)
//
// Warps 0-3 and 4-7 are the two halves' softmax, warp 8 loads (bulk copies of prepared blocks into a ring),
// warp 9 issues, warps 10-15 list the CTA's pieces of work and normalise the next piece's queries.  The halves
// alternate: while one half's S is worked on, the other's PV and the next QK run: PV0(j) QK0(j+1) PV1(j)
// QK1(j+1).  The products of one thread run in order, so QK may write S over the P that the PV ahead of it
// reads, and a half whose S(j) is complete knows that its PV(j-1) is.
//
// Numbers.  S is in units of one factor c (softmax_scale, log2 e and the gains' power of two).  The
// tile's values are 2^-E of themselves, so a row's weights are P_t = 2^(c S_t + E + 7 - m) with m a running
// reference: moved only when the maximum of c S_t + E exceeds it by 2^8, to that maximum less the tile's spread of
// sizes (TileScale: so that a large token that the row does not see, or gives no weight, takes no bits from the
// others).  P <= 2^15 fits fp16, whose normal range then reaches 2^-21 below the largest weight.  The sum of the softmax
// is kept in fp32 from the unrounded weights, 2^-E of each tile's; O, in TMEM, is in fp32.  fp16 instead of bf16 because
// keys and queries are normalised (bounded) and a tile's values have an exponent of their own: 8 times smaller roundings
// at the same rate.  A tile whose latents differ too much holds its values as bf16, and its P is bf16 too.
//
// Work.  A CTA an SM takes an even share of the list of (unit, query tile, token tile); a query tile that is
// cut leaves its parts in the workspace and prefill_join_kernel adds them, by weights 2^(m_s - max m).  Query
// tiles go to the CTAs in turn, so that neighbours work on one unit and share its keys and values in L2: four
// prompts of 4096 tokens took 2468 us with contiguous shares and 2180 so.
//
// Bound: the tensor core.  A token tile takes 24 + 16 products of 128 x 128 x 16 (d_h + d_r = 192, d_v = 128), 64 cycles
// each: 2560; PV's are slower, B in rows of tokens, for 2688.  The steady state takes 3790: shared memory carries each
// product's 4 KB of B, QK's 4 KB of A and the ring's copies, and the softmax chain (load, maximum, exponentials,
// store) of a half has to end within the other half's products.  128 heads, 1024 queries over 16000 tokens: 731 us
// for this kernel, 1.78 PFLOP/s of 1.96 measured for a bf16 library product; 76 % of tensor cycles active.
#include "prefill.cuh"

namespace qkmla {
namespace pf {
namespace {

using namespace tc;

constexpr int kConverters = 6;             // warps that list the work and normalise queries
constexpr int kThreadsA = (10 + kConverters) * 32;
// Registers: 512 threads start with 128 each, the whole register file.  The softmax keeps a row of 128 logits (a loop over
// parts of the row, read twice, took 1029 us where this takes 909, on 1024 queries over 16000 tokens), so each of the
// other warps' two warpgroups gives up 64 a thread and each half's takes as many.
constexpr int kRegsSoftmax = 192, kRegsOther = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsOther <= 4 * 128, "register split");
constexpr int kUnits = 8;                  // ring, in blocks
constexpr int kGroups = 8;                 // barriers of groups (a token tile's key blocks, or its value blocks)

// A piece of work: tiles [t0, t1) of a query tile.
struct Piece {
    int unit;                              // -1: the end
    int t0, t1, nt;                        // nt: tiles of the whole query tile
    int head, gap;                         // tile t is token tile t below head, t + gap from there
    int tile0, skip;                       // and tile0 + t of the workspace, tile0 + t + skip from there
    int n_lo;                              // causal length of the first query
    int queries;
    int row0;                              // first row in q and o
};

struct __align__(16) Shared {
    uint64_t full[kGroups], empty[kGroups];
    uint64_t q_full[2], q_empty[2], q0_full[2];
    uint64_t s_full[2], pa_full[2], pb_full[2], o_full[2];
    uint64_t piece_full[kAhead], piece_empty[kAhead], conv_full[kAhead];
    uint64_t done;
    Piece piece[kAhead];
    int info[4];                           // tinfo of the last token tiles whose keys were issued
    uint32_t tmem;
    int fail;
    int issued;                            // groups whose copies were issued
    int q_issued[2];                       // query halves whose copies were issued
    alignas(16) float gain[192];           // gamma_q gamma_k, then gamma_rope_q, times a power of two
    float factor;                          // of the logits: softmax_scale, log2 e and that power
};
static_assert(sizeof(Shared) <= 2048, "beside the blocks");

template <int DH>
constexpr int smem_bytes() { return (2 * (DH / 64 + 1) + kUnits) * kBlock + 1024 + 2048; }

// One CTA's part of the list.
struct Walk {
    Place at, end = {};
    bool first;

    // The next piece; false at the end.
    __device__ __forceinline__ bool next(const Params& p, Piece& s) {
#pragma unroll 1
        for (;;) {
            if (at.m > end.m || at.m >= p.ctas * p.deep) return false;
            const bool last = at.m == end.m;
            if (last && end.t == 0 && end.nt > 0) return false;
            s.t0 = first ? at.t : 0;
            first = false;
            int j;
            if (!tile_of_place(p, at.m++, s.unit, j)) continue;
            const int4 a = p.qinfo[2 * j], b = p.qinfo[2 * j + 1];
            if (a.x < 0) continue;                         // an unused slot
            s.nt = a.z;
            s.t1 = last ? end.t : s.nt;
            if (s.t0 == s.t1 && s.nt > 0) continue;
            s.head = a.w;
            s.gap = b.x;
            s.n_lo = b.y;
            s.queries = b.z;
            const int4 seq = p.seq[2 * a.x];
            s.skip = s.gap - p.seq[2 * a.x + 1].x;
            s.tile0 = seq.y;
            s.row0 = seq.z + a.y;
            return true;
        }
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// ---- queries ----
// Four rows of a query tile, rt .. rt + 3, eight lanes a row: normalised and times the gains as fp16 to row rt & 127 of
// the half at `dst` (blocks of 64 columns).  Normalised values are at most sqrt d; the gains come with a power of two that
// brings the largest into [1, 2), so that no scale overflows, and what fp16 loses below 2^-14 is 2^-25 of a logit's range.
// A lane's values are 4 of every 32 neighbours.
template <int N>
struct QueryRow {
    uint64_t v[N][2];                      // packed pairs
    __device__ __forceinline__ void load(const void* x, int64_t at, bool bf16, int sub) {
        if (!bf16) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float4 f = *reinterpret_cast<const float4*>((const float*)x + at + (j * 8 + sub) * 4);
                v[j][0] = dec::f2(f.x, f.y);
                v[j][1] = dec::f2(f.z, f.w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint2 u = *reinterpret_cast<const uint2*>((const uint16_t*)x + at + (j * 8 + sub) * 4);
                v[j][0] = dec::f2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
                v[j][1] = dec::f2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
            }
        }
    }
    __device__ __forceinline__ float squares() const {
        uint64_t a = dec::f2_mul(v[0][0], v[0][0]), b = dec::f2_mul(v[0][1], v[0][1]);
#pragma unroll
        for (int j = 1; j < N; ++j) {
            a = dec::f2_fma(v[j][0], v[j][0], a);
            b = dec::f2_fma(v[j][1], v[j][1], b);
        }
        const float2 t = dec::f2_unpack(dec::f2_add(a, b));
        float s = t.x + t.y;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    }
    __device__ __forceinline__ void store(float a, const float* gain, uint8_t* dst, int row, int sub) const {
        const uint64_t a2 = dec::f2(a, a);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int col = (j * 8 + sub) * 4;
            const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(gain + col);
            const float2 lo = dec::f2_unpack(dec::f2_mul(dec::f2_mul(v[j][0], a2), g.x)), hi = dec::f2_unpack(dec::f2_mul(dec::f2_mul(v[j][1], a2), g.y));
            *reinterpret_cast<uint2*>(dst + (col >> 6) * kBlock + sw128_offset(row, col & 63)) = make_uint2(pack_f16(lo.x, lo.y), pack_f16(hi.x, hi.y));
        }
    }
};

template <int DH, int DR>
__device__ __forceinline__ void query_rows(const Params& p, const Piece& s, const float* gain, int rt, uint8_t* dst, int lane) {
    const int sub = lane & 7;
    rt += lane >> 3;
    const int i = rt >> p.hp_log;
    const int64_t row = s.row0 + (i < s.queries ? i : 0), head = (int64_t)s.unit * p.hp + (rt & (p.hp - 1));
    QueryRow<DH / 32> x;
    QueryRow<DR / 32> y;
    x.load(p.q, row * p.q_row + head * p.q_head, p.q_bf16, sub);
    y.load(p.q_rope, row * p.qr_row + head * p.qr_head, p.q_bf16, sub);
    x.store(rsqrtf(x.squares() / DH + p.eps), gain, dst, rt & 127, sub);
    y.store(rsqrtf(y.squares() / DR + p.eps), gain + DH, dst + DH / 64 * kBlock, rt & 127, sub);
}

// ---- softmax of a tile's row: weights in place of logits ----
// 64 columns of the row together with their maximum (a reduction in the load, on sm_103a).
__device__ __forceinline__ void tmem_ld64_max(uint32_t taddr, float* x, float& top) {
    asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x64.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, %64, [%65];"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
          "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]),
          "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]),
          "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31]), "=f"(x[32]), "=f"(x[33]), "=f"(x[34]), "=f"(x[35]), "=f"(x[36]),
          "=f"(x[37]), "=f"(x[38]), "=f"(x[39]), "=f"(x[40]), "=f"(x[41]), "=f"(x[42]), "=f"(x[43]), "=f"(x[44]), "=f"(x[45]),
          "=f"(x[46]), "=f"(x[47]), "=f"(x[48]), "=f"(x[49]), "=f"(x[50]), "=f"(x[51]), "=f"(x[52]), "=f"(x[53]), "=f"(x[54]),
          "=f"(x[55]), "=f"(x[56]), "=f"(x[57]), "=f"(x[58]), "=f"(x[59]), "=f"(x[60]), "=f"(x[61]), "=f"(x[62]), "=f"(x[63]),
          "=f"(top)
        : "r"(taddr));
}
// Bit k: whether the row sees column c0 + k.  It sees columns below `end`, with a window those from `from` on or below
// `sink`.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t seen32(int c0, int end, int from, int sink) {
    return below(end - c0) & (~below(from - c0) | below(sink - c0));
}

// Weights of the row's 128 tokens to TMEM in two halves, each signalled as soon as it lies there.  Returns the sum of the
// unrounded weights.
template <bool BF>
__device__ __forceinline__ float weights_out(float (&x)[128], float c, float off, uint32_t t_s, uint64_t* first, uint64_t* second, int lane) {
    const uint64_t c2 = dec::f2(c, c), off2 = dec::f2(off, off);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 128; k += 32) {
        uint32_t w[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const float2 a = dec::f2_unpack(dec::f2_fma(dec::f2(x[k + 2 * q], x[k + 2 * q + 1]), c2, off2));
            const float u = ex2(a.x), v = ex2(a.y);
            sum[q & 1] = dec::f2_add(sum[q & 1], dec::f2(u, v));
            w[q] = BF ? pack_bf16(u, v) : pack_f16(u, v);
        }
        tmem_st16(t_s + k / 2, w);
        if (k == 32 || k == 96) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(k == 32 ? first : second);
        }
    }
    const float2 s = dec::f2_unpack(dec::f2_add(sum[0], sum[1]));
    return s.x + s.y;
}

template <int DH, int DR, int DV>
__global__ void __launch_bounds__(kThreadsA, 1) prefill_attend_kernel(const __grid_constant__ Params p) {
    constexpr int KU = DH / 64 + 1;                        // blocks of a key tile
    constexpr int VU = DV / 64;
    constexpr int kHalf = KU * kBlock;                     // a half's queries
    constexpr uint32_t kS = 0, kO = 256;                   // TMEM: S of half h at 128 h, O at 256 + 128 h
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    uint8_t* ring = sm + 2 * kHalf;
    Shared* sh = reinterpret_cast<Shared*>(ring + kUnits * kBlock);
    // (the warp's number by a shuffle: the compiler then knows that a role's branches and addresses are the warp's)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int cta = blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < kGroups; ++i) { mbar_init(&sh->full[i], 1); mbar_init(&sh->empty[i], 1); }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(&sh->piece_full[i], 1);
            mbar_init(&sh->piece_empty[i], 10);            // loads, products, eight softmax warps
            mbar_init(&sh->conv_full[i], kConverters);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], 1);
            mbar_init(&sh->q0_full[i], 4);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->pa_full[i], 4);
            mbar_init(&sh->pb_full[i], 4);
            mbar_init(&sh->o_full[i], 1);
            sh->q_issued[i] = 0;
        }
        mbar_init(&sh->done, 1);
        sh->fail = 0;
        sh->issued = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(&sh->tmem, 512);
        tmem_relinquish();
    }
    if (warp == 10) {
        float g[(DH + DR) / 32], top = 0.f;
#pragma unroll
        for (int i = 0; i < (DH + DR) / 32; ++i) {
            const int j = i * 32 + lane;
            g[i] = j < DH ? p.gamma_q[j] * p.gamma_k[j] : p.gamma_rope ? p.gamma_rope[j - DH] : 1.f;
            if (isfinite(g[i])) top = fmaxf(top, fabsf(g[i]));
        }
        top = warp_max(top);
        const int e = top > 0.f ? min(max(ilogbf(top), -100), 100) : 0;
#pragma unroll
        for (int i = 0; i < (DH + DR) / 32; ++i) sh->gain[i * 32 + lane] = g[i] * pow2i(-e);
        if (lane == 0) sh->factor = p.scale_log2 * pow2i(e);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    pdl_wait();
    pdl_trigger();
    const int64_t all = p.pre[p.ctas * p.deep];
    const int n_cta = sharing(p, all);
    const bool busy = all > 0 && cta < n_cta;              // uniform

    if (!busy) {
    } else if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
      if (warp == 8) {
        // ---- loads ----
        if (lane == 0) {
            int group = 0, unit = 0;                       // issued so far
            int freed = 0, freed_units = 0;
            uint32_t qe_phase = 0;                         // bit h
            int last_halves = 0;                           // of the piece ahead, 0 if it has no tiles
            bool ok = true;
#pragma unroll 1
            for (int k = 0; ok; ++k) {
                if (!(ok = wait_or_fail(&sh->piece_full[k % kAhead], (k / kAhead) & 1, &sh->fail))) break;
                const Piece s = sh->piece[k % kAhead];
                if (s.unit < 0) break;
                const int n = s.t1 - s.t0, halves = n == 0 ? 0 : s.queries * p.hp > 128 ? 2 : 1;
                const size_t g = (size_t)((int64_t)s.unit * p.G / p.units), gv = (size_t)((int64_t)s.unit * p.Gv / p.units);
                size_t tile = 0;
                int info_next = n > 0 ? p.tinfo[s.tile0 + (s.t0 < s.head ? s.t0 : s.t0 + s.skip)] : 0;
                // keys and values of a tile in turn, the piece's queries behind the first keys
#pragma unroll 1
                for (int q = 0; q < max(2 * n, 1) && ok; ++q) {
                    const bool value = q & 1;
                    if (n > 0) {
                        const int blocks = value ? VU : KU;
                        if (!value) {
                            const int t = s.t0 + (q >> 1);
                            tile = (size_t)s.tile0 + (t < s.head ? t : t + s.skip);
                            // (through shared memory: a load from L2 in the other warps' loops would be waited for there)
                            sh->info[(group >> 1) & 3] = info_next;
                            if (t + 1 < s.t1) info_next = p.tinfo[s.tile0 + (t + 1 < s.head ? t + 1 : t + 1 + s.skip)];
                        }
                        const uint8_t* src = value ? p.v + (tile * p.Gv + gv) * (size_t)(VU * kBlock) : p.kc + (tile * p.G + g) * (size_t)((KU - 1) * kBlock);
#pragma unroll 1
                        while (ok && unit + blocks - kUnits > freed_units) {
                            ok = wait_or_fail(&sh->empty[freed % kGroups], (freed / kGroups) & 1, &sh->fail);
                            freed_units += (freed & 1) ? VU : KU;
                            ++freed;
                        }
                        if (!ok) break;
                        uint64_t* bar = &sh->full[group % kGroups];
                        mbar_arrive_expect_tx(bar, blocks * kBlock);
#pragma unroll 1
                        for (int i = 0; i < blocks; ++i, ++unit)
                            bulk_load(ring + (unit % kUnits) * kBlock, !value && i == KU - 1 ? p.krope + tile * kBlock : src + (size_t)i * kBlock, kBlock, bar);
                        ++group;
                        *(volatile int*)&sh->issued = group;
                    }
                    if (q > 0) continue;
                    // Every piece's conversion is waited for, of one without tiles too: piece_empty then says that all converting
                    // warps have been through the piece, so that none falls a phase of either barrier behind.  (The first
                    // piece's rows go to shared memory directly.)
                    if (k > 0) ok = wait_or_fail(&sh->conv_full[k % kAhead], ((k - 1) / kAhead) & 1, &sh->fail);
                    // a query half is read by the products until the last ones of the piece ahead have ended
#pragma unroll 1
                    for (int h = 0; h < 2 && ok; ++h) {
                        if (h < last_halves) {
                            ok = wait_or_fail(&sh->q_empty[h], (qe_phase >> h) & 1, &sh->fail);
                            qe_phase ^= 1u << h;
                        }
                        if (!ok || h >= halves || k == 0) continue;
                        mbar_arrive_expect_tx(&sh->q_full[h], kHalf);
                        bulk_load(sm + h * kHalf, p.qs + ((size_t)(kAhead * cta + k % kAhead) * 2 + h) * kHalf, kHalf, &sh->q_full[h]);
                        *(volatile int*)&sh->q_issued[h] = *(volatile int*)&sh->q_issued[h] + 1;
                    }
                    if (k > 0) mbar_arrive(&sh->piece_empty[(k - 1) % kAhead]);     // the converted rows of piece k - 1 are no longer read
                    last_halves = halves;
                }
            }
        }
        __syncwarp();
      } else if (warp == 9) {
        // ---- products ----
        if (elect_one()) {
        constexpr uint32_t bf = (1u << 7) | (1u << 10);
        constexpr uint32_t id_s = idesc_bf16(128, 128, 0, 0) & ~bf;
        constexpr uint32_t id_o = idesc_bf16(128, DV, 0, 1) & ~bf;
        // descriptors are formed once and moved by offsets: the issue has to keep up with 65 cycles a product
        constexpr uint32_t kStep = kBlock >> 4;
        const uint32_t q_desc = desc_low(sm, 16);
        const uint32_t k_desc = desc_low(ring, 16);
        const uint32_t v_desc = desc_low(ring, kBlock / 2);   // 64 tokens, 64-column boxes 8 KB apart
        int group = 0, unit = 0, k = 0;                    // groups and blocks consumed, pieces fetched
        uint32_t p_phase = 0, q_phase = 0;                 // bit h (arrays would lie in local memory)
        int halves = 0, left = 0, q_at = 0;                // of the piece whose logits come next: tiles left, its place in the queue
        int cur = 0;                                       // halves whose weights are awaited
        bool cur_first = false, cur_last = false;
        // A round: for each half, O += P V of the tile whose weights are awaited, then S of the next tile (of the
        // same piece or of the next one).
        for (;;) {
            bool first = false;
            // the next piece (halves -1: there is none); with weights awaited no more than one, which may have no tiles:
            // the one behind it is not listed before they have been used
            while (left == 0 && halves >= 0) {
                if (!wait_or_fail(&sh->piece_full[k % kAhead], (k / kAhead) & 1, &sh->fail)) goto give_up;
                const Piece& s = sh->piece[k % kAhead];
                if (s.unit < 0) { halves = -1; break; }
                left = s.t1 - s.t0;
                halves = s.queries * p.hp > 128 ? 2 : 1;
                first = true;
                q_at = k;
                mbar_arrive(&sh->piece_empty[k % kAhead]);
                ++k;
                if (cur > 0) break;
            }
            const int nxt = left > 0 ? halves : 0;
            if (cur == 0 && nxt == 0) break;
            const int gv = group, gk = group + (cur > 0 ? 1 : 0);
            const bool as_bf = (sh->info[(gv >> 1) & 3] & 256) != 0;
            const uint32_t fmt = as_bf ? bf : 0u;
            if (cur == 2 && nxt == 2 && !first) {
                // The same rounds in a straight line, to the piece's end.  The unit takes six or so products ahead; each
                // barrier is looked at, and the next round's operands are formed, while products are still being taken (a
                // wait that succeeds at once costs as much as two of them).
                auto value = [&](int u) { return v_desc + (uint32_t)((u % kUnits) * kStep); };
                uint32_t v0 = value(unit), v1 = VU == 2 ? value(unit + 1) : v0 + kStep / 2, kd[KU];
#pragma unroll
                for (int blk = 0; blk < KU; ++blk) kd[blk] = k_desc + (uint32_t)(((unit + VU + blk) % kUnits) * kStep);
                uint32_t acc = cur_first ? 0u : 1u, id = id_o | fmt;
                uint64_t *b_v = &sh->full[gv % kGroups], *b_k = &sh->full[gk % kGroups], *f_v = &sh->empty[gv % kGroups], *f_k = &sh->empty[gk % kGroups];
                uint32_t ph_v = (gv / kGroups) & 1, ph_k = (gk / kGroups) & 1, ph = p_phase & 1;       // (both halves' phases are alike in a piece of two)
                uint32_t ph1 = (p_phase >> 1) & 1;
                group = gk + 1;
                unit += VU + KU;
                bool seen_a = false, seen_v = false, seen_1 = false;
                for (;;) {
                    uint32_t v0n, v1n, kn[KU];
                    uint64_t *b_vn, *b_kn, *f_vn, *f_kn;
                    uint32_t ph_vn, ph_kn, idn;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t o = tmem + kO + h * 128, a = tmem + kS + h * 128, d = a;
                        const uint32_t php = h ? ph1 : ph;
                        if (!(h == 0 ? seen_a : seen_1) && !wait_or_fail(&sh->pa_full[h], php, &sh->fail)) goto give_up;
                        if (h == 0 && !seen_v && !wait_or_fail(b_v, ph_v, &sh->fail)) goto give_up;
                        tc_fence_after();
                        mma_ts(o, a, v0, id, acc);
                        mma_ts(o, a + 8, v0 + 128, id, 1u);
                        const bool seen_b = mbar_test_wait(&sh->pb_full[h], php);
                        mma_ts(o, a + 16, v0 + 256, id, 1u);
                        mma_ts(o, a + 24, v0 + 384, id, 1u);
                        if (!seen_b && !wait_or_fail(&sh->pb_full[h], php, &sh->fail)) goto give_up;
                        tc_fence_after();
                        mma_ts(o, a + 32, v1, id, 1u);
                        mma_ts(o, a + 40, v1 + 128, id, 1u);
                        bool seen_k = true;
                        if (h == 0) seen_k = mbar_test_wait(b_k, ph_k);
                        mma_ts(o, a + 48, v1 + 256, id, 1u);
                        mma_ts(o, a + 56, v1 + 384, id, 1u);
                        if (h == 1) mma_commit(f_v);
                        if (!seen_k && !wait_or_fail(b_k, ph_k, &sh->fail)) goto give_up;
#pragma unroll
                        for (int blk = 0; blk < KU; ++blk) {
                            if (blk == KU - 1) {            // one more block of products to come
                                if (h == 0) {
                                    seen_1 = mbar_test_wait(&sh->pa_full[1], ph1);
                                } else {
                                    const int gn = group, kg = group + 1;
                                    v0n = value(unit);
                                    v1n = VU == 2 ? value(unit + 1) : v0n + kStep / 2;
#pragma unroll
                                    for (int q = 0; q < KU; ++q) kn[q] = k_desc + (uint32_t)(((unit + VU + q) % kUnits) * kStep);
                                    b_vn = &sh->full[gn % kGroups];
                                    b_kn = &sh->full[kg % kGroups];
                                    f_vn = &sh->empty[gn % kGroups];
                                    f_kn = &sh->empty[kg % kGroups];
                                    ph_vn = (gn / kGroups) & 1;
                                    ph_kn = (kg / kGroups) & 1;
                                    idn = id_o | ((sh->info[(gn >> 1) & 3] & 256) ? bf : 0u);
                                    seen_a = mbar_test_wait(&sh->pa_full[0], ph ^ 1);
                                    seen_v = mbar_test_wait(b_vn, ph_vn);
                                }
                            }
#pragma unroll
                            for (int kk = 0; kk < (blk < KU - 1 ? 4 : DR / 16); ++kk)
                                mma_ss(d, q_desc + (uint32_t)((h * KU + blk) * kStep + kk * 2), kd[blk] + (uint32_t)(kk * 2), id_s, (blk > 0 || kk > 0) ? 1u : 0u);
                        }
                        mma_commit(&sh->s_full[h]);
                        if (left == 1) mma_commit(&sh->q_empty[h]);
                    }
                    mma_commit(f_k);
                    ph ^= 1;
                    ph1 ^= 1;
                    acc = 1u;
                    if (--left == 0) break;
                    v0 = v0n;
                    v1 = v1n;
#pragma unroll
                    for (int q = 0; q < KU; ++q) kd[q] = kn[q];
                    b_v = b_vn; b_k = b_kn; f_v = f_vn; f_k = f_kn;
                    ph_v = ph_vn; ph_k = ph_kn; id = idn;
                    group += 2;
                    unit += VU + KU;
                }
                p_phase = ph | ph1 << 1;
                cur_first = false;
                cur_last = true;
                continue;
            }
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (h < cur) {
                    const uint32_t o = tmem + kO + h * 128, a = tmem + kS + h * 128;
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) { // 64 tokens each
                        if (!wait_or_fail(part ? &sh->pb_full[h] : &sh->pa_full[h], (p_phase >> h) & 1, &sh->fail)) goto give_up;
                        if (h + part == 0 && !wait_or_fail(&sh->full[gv % kGroups], (gv / kGroups) & 1, &sh->fail)) goto give_up;
                        tc_fence_after();
                        const uint32_t v = v_desc + (uint32_t)(VU == 2 ? ((unit + part) % kUnits) * kStep : (unit % kUnits) * kStep + part * (kStep / 2));
#pragma unroll 1
                        for (int i = 0; i < 4; ++i)
                            mma_ts(o, a + part * 32 + i * 8, v + (uint32_t)(i * 128), id_o | fmt, (!cur_first || part > 0 || i > 0) ? 1u : 0u);
                    }
                    p_phase ^= 1u << h;
                    if (h == cur - 1) mma_commit(&sh->empty[gv % kGroups]);
                    if (cur_last) mma_commit(&sh->o_full[h]);
                }
                if (h < nxt) {
                    if (h == 0 && !wait_or_fail(&sh->full[gk % kGroups], (gk / kGroups) & 1, &sh->fail)) goto give_up;
                    if (first) {
                        if (q_at == 0) {
                            if (!wait_or_fail(&sh->q0_full[h], 0, &sh->fail)) goto give_up;
                        } else {
                            if (!wait_or_fail(&sh->q_full[h], (q_phase >> h) & 1, &sh->fail)) goto give_up;
                            q_phase ^= 1u << h;
                        }
                    }
                    tc_fence_after();
                    const int u = unit + (cur > 0 ? VU : 0);
                    const uint32_t d = tmem + kS + h * 128;
#pragma unroll 1
                    for (int blk = 0; blk < KU; ++blk) {
                        const uint32_t kd = k_desc + (uint32_t)(((u + blk) % kUnits) * kStep), qd = q_desc + (uint32_t)((h * KU + blk) * kStep);
#pragma unroll 1
                        for (int kk = 0; kk < (blk < KU - 1 ? 4 : DR / 16); ++kk)
                            mma_ss(d, qd + (uint32_t)(kk * 2), kd + (uint32_t)(kk * 2), id_s, (blk > 0 || kk > 0) ? 1u : 0u);
                    }
                    mma_commit(&sh->s_full[h]);
                    if (left == 1) mma_commit(&sh->q_empty[h]);
                    if (h == nxt - 1) mma_commit(&sh->empty[gk % kGroups]);
                }
            }
            group = gk + (nxt > 0 ? 1 : 0);
            unit += (cur > 0 ? VU : 0) + (nxt > 0 ? KU : 0);
            cur = nxt;
            cur_first = first;
            cur_last = left == 1;
            left -= nxt > 0 ? 1 : 0;
        }
give_up:
        mma_commit(&sh->done);
        }
        __syncwarp();
      } else {
        // ---- the list, and the queries of every piece but the first ----
        Walk walk;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            walk.at = walk.end;
            walk.end = place_of(p, share_start(all, n_cta, cta + i), all);
        }
        walk.first = true;
        if (warp == 10 && lane == 0) {                     // for the join
            p.cuts[cta] = make_int4(walk.at.m, walk.at.t, walk.at.nt, 0);
            if (cta == n_cta - 1) p.cuts[n_cta] = make_int4(walk.end.m, walk.end.t, walk.end.nt, 0);
        }
        bool ok = true;
#pragma unroll 1
        for (int k = 0;; ++k) {
            Piece s;
            if (!walk.next(p, s)) s.unit = -1;
            if (k > 0 && s.unit >= 0 && s.t0 < s.t1) {
                // the raw rows into L2: reading them then takes its latency
                const int row_bytes = p.q_bf16 ? 2 * DH : 4 * DH, rope_bytes = p.q_bf16 ? 2 * DR : 4 * DR, esz = p.q_bf16 ? 2 : 4;
#pragma unroll 1
                for (int rt = (warp - 10) * 32 + lane; rt < min(s.queries * p.hp, kRowsQ); rt += kConverters * 32) {
                    const int64_t row = s.row0 + (rt >> p.hp_log), head = (int64_t)s.unit * p.hp + (rt & (p.hp - 1));
                    const char* x = (const char*)p.q + (row * p.q_row + head * p.q_head) * esz;
                    const char* y = (const char*)p.q_rope + (row * p.qr_row + head * p.qr_head) * esz;
#pragma unroll 1
                    for (int i = 0; i < row_bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + i));
#pragma unroll 1
                    for (int i = 0; i < rope_bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(y + i));
                }
            }
            if (k >= kAhead) ok = wait_long(&sh->piece_empty[k % kAhead], (k / kAhead - 1) & 1, &sh->fail);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (warp == 10 && lane == 0) {
                sh->piece[k % kAhead] = s;
                mbar_arrive(&sh->piece_full[k % kAhead]);
            }
            if (s.unit < 0) break;
            if (k == 0) continue;
            if (s.t0 < s.t1) {
                const int rows = min(s.queries * p.hp, kRowsQ);
                uint8_t* dst = p.qs + (size_t)(kAhead * cta + k % kAhead) * (2 * kHalf);
#pragma unroll 1
                for (int rt = (warp - 10) * 4; rt < rows; rt += kConverters * 4) query_rows<DH, DR>(p, s, sh->gain, rt, dst + (rt >> 7) * kHalf, lane);
                asm volatile("fence.proxy.async.global;" ::: "memory");
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->conv_full[k % kAhead]);
        }
      }
    } else {
        // ---- softmax: thread = row ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int h = warp >> 2, rt = tid;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t t_s = tmem + lane_base + kS + h * 128, t_o = tmem + lane_base + kO + h * 128;
        const int* we = reinterpret_cast<const int*>(p.weights);
        uint32_t s_phase = 0, o_phase = 0;
        int tiles = 0;                                                  // token tiles of the CTA so far
        const float c = sh->factor;
        bool ok = true;
#pragma unroll 1
        for (int k = 0;; ++k) {
            ok = wait_or_fail(&sh->piece_full[k % kAhead], (k / kAhead) & 1, &sh->fail);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const Piece& s = sh->piece[k % kAhead];                          // (read where it is needed: registers are few)
            if (s.unit < 0) break;
            const bool mine = h == 0 || s.queries * p.hp > 128;         // uniform in a warp
            if (mine && k == 0 && s.t0 < s.t1) {
                // the first piece's queries, straight to shared memory: a warp its own 32 rows
#pragma unroll 1
                for (int q = 0; q < 32; q += 4) query_rows<DH, DR>(p, s, sh->gain, warp * 32 + q, sm + h * kHalf, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->q0_full[h]);
            }
            const int i = rt >> p.hp_log;                               // the row's query within the tile
            const bool there = i < s.queries;
            const int n_row = there ? s.n_lo + i : 0;                   // causal length
            float m = -INFINITY, sum = 0.f;
            auto tile_at = [&](int t) { return t < s.head ? t : t + s.gap; };
            if (!mine) tiles += s.t1 - s.t0;
#pragma unroll 1
            for (int t = s.t0; t < s.t1 && mine; ++t, ++tiles) {
                const int first = tile_at(t) * kTile;
                // tiles that some row does not see whole (uniform over the tile's rows)
                const bool edge = first + kTile > s.n_lo || (p.window > 0 && first < s.n_lo + s.queries - 1 - p.window && first + kTile > p.sinks);
                ok = wait_or_fail(&sh->s_full[h], s_phase, &sh->fail);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                s_phase ^= 1;
                tc_fence_after();
                const int info = sh->info[tiles & 3], e = (info & 255) - 64;
                const bool as_bf = (info & 256) != 0;
                if (edge) {
                    // hidden logits to -inf, in place: a rolled loop of 16 columns
                    const int end = n_row - first, from = p.window > 0 ? end - p.window : 0, sink = p.window > 0 ? p.sinks - first : 0;
#pragma unroll 1
                    for (int q = 0; q < 128; q += 32) {
                        uint32_t seen = seen32(q, end, from, sink);
#pragma unroll 1
                        for (int r = 0; r < 32; r += 16, seen >>= 16) {
                            if (__all_sync(0xffffffffu, (seen & 0xffffu) == 0xffffu)) continue;
                            uint32_t v[16];
                            tmem_ld16(t_s + q + r, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i2 = 0; i2 < 16; ++i2) v[i2] = seen >> i2 & 1 ? v[i2] : 0xff800000u;
                            tmem_st16(t_s + q + r, v);
                        }
                    }
                    tmem_wait_st();
                }
                float x[128], top, top2;
                tmem_ld64_max(t_s, x, top);
                tmem_ld64_max(t_s + 64, x + 64, top2);
                tmem_wait_ld();
                top = fmaxf(top, top2);
                const float cand = fmaf(top, c, (float)e);
                const bool move = cand > m + 8.f;
                if (__any_sync(0xffffffffu, move)) {
                    const float m2 = move ? cand - (float)(info >> 9) : m;
                    const float a = move ? ex2(m - m2) : 1.f;           // 0 while nothing was seen
                    sum *= a;
                    if (t > s.t0) {
#pragma unroll 1
                        for (int q = 0; q < DV; q += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + q, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int r = 0; r < 16; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * a);
                            tmem_st16(t_o + q, o);
                        }
                    }
                    m = m2;
                }
                const float off = (float)(e + 7) - (m == -INFINITY ? 0.f : m);
                const float part = as_bf ? weights_out<true>(x, c, off, t_s, &sh->pa_full[h], &sh->pb_full[h], lane)
                                         : weights_out<false>(x, c, off, t_s, &sh->pa_full[h], &sh->pb_full[h], lane);
                sum = fmaf(part, pow2i(-e), sum);
            }
            if (!mine) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->piece_empty[k % kAhead]);
                continue;
            }
            if (s.t0 < s.t1 && ok) ok = wait_or_fail(&sh->o_full[h], o_phase, &sh->fail);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (s.t0 < s.t1) {
                o_phase ^= 1;
                tc_fence_after();
            }
            // the row's output, or its part's fp32 sums and, for the join, reference and sum
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            const int gv = (int)((int64_t)s.unit * p.Gv / p.units);
            const float inv = !whole ? 1.f : sum == 0.f ? 0.f : ldexpf(1.f / sum, we[p.G + gv]);
            const size_t part = (size_t)(2 * cta + (s.t0 > 0 ? 0 : 1)) * kRowsQ;
            // (row r of the tile: query r / hp, head r % hp of the unit)
            auto out = [&](int r) { return ((int64_t)s.row0 + (r >> p.hp_log)) * p.H + s.unit * p.hp + (r & (p.hp - 1)); };
            const bool narrow = whole && !p.o_f32;
            const int r0 = rt & ~3;
#pragma unroll 1
            for (int q = 0; q < DV; q += narrow ? 64 : 32) {
                uint32_t h[4][8];
                // 16 columns a piece as bf16, 8 as fp32; columns from q on
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[16];
                    if (s.t0 < s.t1) {
                        if (narrow) tmem_ld16(t_o + q + c * 16, o);
                        else if (c < 2) tmem_ld16(t_o + q + c * 16, o);
                        tmem_wait_ld();
                    }
                    if (narrow) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            h[c][i] = inv == 0.f ? 0u : pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                    } else if (c < 2) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) h[2 * c + (i >> 3)][i & 7] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
                    }
                }
                quad_transpose(h, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = r0 + k;
                    if ((r >> p.hp_log) >= s.queries) continue;
                    uint8_t* dst = narrow ? (uint8_t*)((uint16_t*)p.o + out(r) * DV + q) : whole ? (uint8_t*)((float*)p.o + out(r) * DV + q)
                                                                                                : (uint8_t*)(p.part_o + (part + r) * DV + q);
                    const uint32_t (&one)[8] = h[k];
                    st_global_v8(dst + (lane & 3) * 32, {one[0], one[1], one[2], one[3]}, {one[4], one[5], one[6], one[7]});
                }
            }
            if (there) {
                if (!whole) p.part_ml[part + rt] = make_float2(m, sum);
                else if (p.lse) p.lse[out(rt)] = sum == 0.f ? -INFINITY : (m - 7.f) * kLn2 + logf(sum);
            }
            tc_fence_before();                                          // the next tile's PV writes O after this half's P
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->piece_empty[k % kAhead]);
        }
    }
    __syncthreads();
    if (busy) {
        // a CTA that gave up waits for its copies in flight, and always for its products
        wait_or_fail(&sh->done, 0, &sh->fail);
        if (*(volatile int*)&sh->fail && tid == 0) {
            report(p.status, QKMLA_ERR_TIMEOUT);
            const int n = *(volatile int*)&sh->issued;
            for (int g = max(0, n - kGroups); g < n; ++g) dec::wait_bounded(&sh->full[g % kGroups], (g / kGroups) & 1, p.status);
            for (int h = 0; h < 2; ++h) {
                const int q = *(volatile int*)&sh->q_issued[h];
                if (q > 0) dec::wait_bounded(&sh->q_full[h], (q - 1) & 1, p.status);
            }
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
// Bound: latency (each row's parts and their references are found, then read): 151 cut tiles of 256 x 128 values, 49 MB,
// take 24 us with a cold L2 and less behind the attention, which leaves the parts there.
constexpr int kThreadsJ = 128;
constexpr int kRowsJ = 16;

template <int DV>
__global__ void __launch_bounds__(kThreadsJ) prefill_join_kernel(const __grid_constant__ Params p) {
    pdl_wait();
    pdl_trigger();
    const int64_t all = p.pre[p.ctas * p.deep];
    const int n_cta = sharing(p, all);
    const int k = blockIdx.x + 1;
    if (all == 0 || k >= n_cta) return;
    __shared__ Place places[kMaxCtas + 1];
    __shared__ int parts[kMaxCtas];
    __shared__ int count;
    for (int q = k - 1 + threadIdx.x; q <= n_cta; q += kThreadsJ) {
        const int4 c = p.cuts[q];
        places[q] = Place{c.x, c.y, c.z};
    }
    __syncthreads();
    const Place at = places[k];
    if (!at.inside()) return;
    if (k > 1) {
        const Place prev = places[k - 1];
        if (prev.inside() && prev.m == at.m) return;
    }
    // parts: CTA k - 1's last piece, then the first pieces of CTAs k .. last - 1 (one that got no tile has none)
    if (threadIdx.x == 0) {
        parts[0] = 2 * (k - 1) + 1;
        int n = 1;
        for (int q = k; q < n_cta; ++q) {
            const Place to = places[q + 1];
            const bool same = to.m == at.m && to.t < at.nt;
            if (!(same && to.t == places[q].t)) parts[n++] = 2 * q;
            if (!same) break;
        }
        count = n;
    }
    __syncthreads();
    const int n = count;
    int unit, j;
    tile_of_place(p, at.m, unit, j);
    const int4 a = p.qinfo[2 * j], b = p.qinfo[2 * j + 1];
    const int4 seq = p.seq[2 * a.x];
    const int gv = (int)((int64_t)unit * p.Gv / p.units);
    const int e = reinterpret_cast<const int*>(p.weights)[p.G + gv];
    constexpr int kLanes = DV / 4;                          // lanes a row, 4 values each
    constexpr int kPerPass = kThreadsJ / kLanes;
#pragma unroll 1
    for (int q = threadIdx.x / kLanes; q < kRowsJ; q += kPerPass) {
        const int rt = blockIdx.y * kRowsJ + q, i = rt / p.hp;
        if (i >= b.z) continue;
        float top = -INFINITY;
#pragma unroll 4
        for (int s = 0; s < n; ++s) top = fmaxf(top, p.part_ml[(size_t)parts[s] * kRowsQ + rt].x);
        float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        const int col = threadIdx.x % kLanes * 4;
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const size_t row = (size_t)parts[s] * kRowsQ + rt;
            const float2 ml = p.part_ml[row];
            // a part that saw nothing has m = -inf and weight 0, unless its sum is NaN (a key that is not finite)
            const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - top);
            const float4 v = *reinterpret_cast<const float4*>(p.part_o + row * DV + col);
            sum = fmaf(w, ml.y, sum);
            o[0] = fmaf(w, v.x, o[0]); o[1] = fmaf(w, v.y, o[1]); o[2] = fmaf(w, v.z, o[2]); o[3] = fmaf(w, v.w, o[3]);
        }
        const int head = unit * p.hp + rt % p.hp;
        const int64_t r = seq.z + a.y + i;
        const float inv = sum == 0.f ? 0.f : ldexpf(1.f / sum, e);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = sum == 0.f ? 0.f : o[c] * inv;
        const int64_t to = (r * p.H + head) * DV + col;
        if (p.o_f32) *reinterpret_cast<float4*>((float*)p.o + to) = make_float4(o[0], o[1], o[2], o[3]);
        else *reinterpret_cast<uint2*>((uint16_t*)p.o + to) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
        if (col == 0 && p.lse) p.lse[r * p.H + head] = sum == 0.f ? -INFINITY : (top - 7.f) * kLn2 + logf(sum);
    }
}

template <int DH, int DR, int DV>
int launch(const Params& p, cudaStream_t s) {
    auto k = prefill_attend_kernel<DH, DR, DV>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<DH>()) != cudaSuccess) return QKMLA_ERR_CUDA;
    if (launch_pdl(k, dim3(p.ctas), dim3(kThreadsA), smem_bytes<DH>(), s, p) != cudaSuccess) return QKMLA_ERR_CUDA;
    if (p.ctas < 2) return QKMLA_OK;
    return launch_pdl(prefill_join_kernel<DV>, dim3(p.ctas - 1, kRowsQ / kRowsJ), dim3(kThreadsJ), 0, s, p) == cudaSuccess ? QKMLA_OK
                                                                                                                         : QKMLA_ERR_CUDA;
}

template <int DH, int DR>
int launch_dv(const Params& p, cudaStream_t s) { return p.d_v == 128 ? launch<DH, DR, 128>(p, s) : launch<DH, DR, 64>(p, s); }

}  // namespace

int launch_attend(const Params& p, cudaStream_t s) {
    if (p.d_h == 128) return p.d_r == 64 ? launch_dv<128, 64>(p, s) : launch_dv<128, 32>(p, s);
    return p.d_r == 64 ? launch_dv<64, 64>(p, s) : launch_dv<64, 32>(p, s);
}

}  // namespace pf
}  // namespace qkmla

using namespace qkmla;

namespace {

int check_sizes(const qkmla_prefill_args* a) {
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
    return QKMLA_OK;
}

int check_pointers(const qkmla_prefill_args* a) {
    const bool q8 = a->cache_dtype == QKMLA_E4M3;
    if (q8 != (a->kv_scale != nullptr)) return QKMLA_ERR_INVALID;
    for (int64_t st : {a->q_row_stride, a->q_head_stride, a->qr_row_stride, a->qr_head_stride})
        if (st % 4) return QKMLA_ERR_INVALID;
    if (!a->q || !a->q_rope || !a->gamma_q || !a->gamma_k || !a->weights || !a->kv_cache || !a->ak_cache || !a->chunk_start ||
        !a->seq_lens || !a->o)
        return QKMLA_ERR_INVALID;
    if ((uintptr_t)a->o % 32) return QKMLA_ERR_INVALID;
    for (const void* ptr : {a->q, a->q_rope, a->weights, a->kv_cache})
        if ((uintptr_t)ptr % 16) return QKMLA_ERR_INVALID;
    for (const void* ptr : {(const void*)a->gamma_q, (const void*)a->gamma_k, (const void*)a->gamma_rope_q, (const void*)a->kv_scale,
                            (const void*)a->chunk_start, (const void*)a->seq_lens, (const void*)a->page_table, (const void*)a->lse})
        if ((uintptr_t)ptr % 4) return QKMLA_ERR_INVALID;
    if ((uintptr_t)a->ak_cache % ((a->flags & QKMLA_FLAG_ALPHA_F16) ? 2 : 4)) return QKMLA_ERR_INVALID;
    if (!a->workspace) return QKMLA_ERR_WORKSPACE;
    if ((uintptr_t)a->workspace % 256) return QKMLA_ERR_INVALID;
    return QKMLA_OK;
}

// Everything that follows from the (checked) arguments; the workspace's parts from a->workspace on.
int make_params(const qkmla_prefill_args* a, pf::Params* p, size_t* bytes) {
    const int units = a->G > a->G_v ? a->G : a->G_v, hp = a->H / units;
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
    p->q_bf16 = a->q_dtype == QKMLA_BF16;
    p->o_f32 = a->o_dtype == QKMLA_F32;
    p->ak_f16 = (a->flags & QKMLA_FLAG_ALPHA_F16) ? 1 : 0;
    p->total_tokens = a->total_tokens;
    p->units = units;
    p->hp = hp;
    while ((1 << p->hp_log) < hp) ++p->hp_log;
    p->tq = pf::kRowsQ / hp;
    p->nq = a->rows / p->tq + a->B;
    p->max_tiles = (int)(a->total_tokens / pf::kTile) + a->B;
    p->ctas = device_sm_count();
    if (p->ctas <= 0) return QKMLA_ERR_CUDA;
    if (p->ctas > pf::kMaxCtas) p->ctas = pf::kMaxCtas;
    p->deep = (int)(((int64_t)units * p->nq + p->ctas - 1) / p->ctas);
    uintptr_t at = (uintptr_t)a->workspace;
    auto take = [&](size_t n) {
        const uintptr_t r = at;
        at += (n + 255) & ~(size_t)255;
        return r;
    };
    const size_t tiles = p->max_tiles, nq = p->nq;
    p->seq = (int4*)take(sizeof(int4) * 2 * a->B);
    p->qinfo = (int4*)take(sizeof(int4) * 2 * nq);
    p->pre = (int64_t*)take(8 * ((size_t)p->ctas * p->deep + 1));
    p->cuts = (int4*)take(sizeof(int4) * (p->ctas + 1));
    p->tinfo = (int*)take(4 * tiles);
    p->part_ml = (float2*)take(sizeof(float2) * 2 * p->ctas * pf::kRowsQ);
    p->part_o = (float*)take(4 * (size_t)2 * p->ctas * pf::kRowsQ * a->d_v);
    p->krope = (uint8_t*)take(tiles * pf::kBlock);
    p->kc = (uint8_t*)take(tiles * a->G * (a->d_h / 64) * pf::kBlock);
    p->v = (uint8_t*)take(tiles * a->G_v * (a->d_v / 64) * pf::kBlock);
    p->qs = (uint8_t*)take((size_t)p->ctas * 2 * pf::kAhead * (a->d_h / 64 + 1) * pf::kBlock);
    *bytes = at - (uintptr_t)a->workspace;
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
    return QKMLA_OK;
}

}  // namespace

extern "C" size_t qkmla_prefill_workspace_size(const qkmla_prefill_args* a) {
    pf::Params p;
    size_t bytes = 0;
    return check_sizes(a) == QKMLA_OK && make_params(a, &p, &bytes) == QKMLA_OK ? bytes : 0;
}

extern "C" int qkmla_prefill(const qkmla_prefill_args* a, void* stream) {
    int rc = check_sizes(a);
    if (rc != QKMLA_OK || a->rows == 0) return rc;
    if ((rc = check_pointers(a)) != QKMLA_OK) return rc;
    pf::Params p;
    size_t bytes = 0;
    if ((rc = make_params(a, &p, &bytes)) != QKMLA_OK) return rc;
    if (a->workspace_bytes < bytes) return QKMLA_ERR_WORKSPACE;
    p.status = device_status_ptr();
    cudaStream_t s = (cudaStream_t)stream;
    if ((rc = pf::launch_expand(p, a->cache_dtype == QKMLA_E4M3, s)) != QKMLA_OK) return rc;
    return pf::launch_attend(p, s);
}
