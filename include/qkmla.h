/*
 * qkmla.h -- C ABI of the QK-Normed MLA decode library (GB300, sm_103a).
 *
 * The method (arXiv 2606.16310, "QK-Normed MLA: QK normalization without full
 * key caching"; gist.science Technical Summary, Methodology) splits
 * post-projection RMSNorm(z) = z * gamma / S(z) into a static weight and a
 * dynamic scalar.  The static key weight gamma_k (with gamma_q) is absorbed
 * into the query; the dynamic key statistic is cached as one inverse-RMS
 * scalar alpha^k per token and KV group next to the MLA latent c_t; decode
 * computes the row/column-scaled logit
 *
 *     l_{i,t,h} = scale * ( alpha^q_{i,h} * alpha^k_{t,g(h)} * (q~_{i,h} . c_t)
 *                           + q^rope_{i,h} . k^rope_t )
 *
 * then a softmax over t and the latent-space output o = sum_t p_t c_t.
 *
 * Three calls form the decode path: qkmla_absorb_query, qkmla_append,
 * qkmla_decode.  Conventions shared by every call:
 *
 *  - All array pointers are DEVICE pointers owned by the caller; the library
 *    keeps no reference after the call returns.  `stream` is a cudaStream_t
 *    (NULL = legacy default stream).  Calls are asynchronous on that stream.
 *  - Host-side validation (null pointers, sizes, dtypes, alignment) returns an
 *    error code before anything is launched.  Launch failures return
 *    QKMLA_ERR_CUDA.  Problems that only the device can see (an out-of-range
 *    page id, a sequence length outside its bounds, an expired bounded wait)
 *    never trap: the kernel skips the offending work and records the first
 *    such error in a per-device status word read by qkmla_get_device_status().
 *  - Shapes: B sequences, s_q query tokens per sequence in this step
 *    (rows = B*s_q), H query heads, G KV groups with g(h) = h / (H/G),
 *    d_h head dim of the content (nope) part, d_c latent dim, d_r RoPE dim.
 *  - Cache: one flat array of slots.  kv_cache[slot] = [c_t (d_c) | k^rope_t
 *    (d_r)] in the cache dtype; ak_cache[slot] = [alpha^k_{t,0..G-1}] fp32
 *    (fp16 with QKMLA_FLAG_ALPHA_F16).
 *    Token t of sequence b lives in slot
 *        page_table[b*max_pages + t/page_size]*page_size + t%page_size,
 *    and with page_table == NULL in slot (b*max_pages + t/page_size)*page_size
 *    + t%page_size (a contiguous cache of max_pages*page_size slots per
 *    sequence).
 *  - The library is stateless apart from the status word and a small per-
 *    device table of launch limits; it is thread-safe.
 *  - Every kernel is launched with programmatic stream serialization and lets
 *    the next kernel of the stream launch early, but for those of qkmla_rope and
 *    qkmla_read_cache, which are waited for in full: what they write may be an
 *    append's new tokens.  A kernel's writes, and its reads of anything another
 *    kernel of this library produces (q~, alpha^q, the cache, q and q_rope of
 *    qkmla_project_query, o), wait for the previous kernel of the stream.  Reads
 *    of inputs no kernel of the library writes, or only those two, may start
 *    earlier: seq_lens in qkmla_decode and qkmla_decode_ext; W^K, the new tokens,
 *    their slots and positions in qkmla_append, qkmla_append_rope and
 *    qkmla_append_q8; out_start, first and the page table in qkmla_read_cache; W^K
 *    and W^V in qkmla_prefill_pack_weights.  A previous kernel that itself signals
 *    early dependent launch must therefore not be writing those inputs (kernels
 *    that do not signal it, and copies, are waited for in full as usual).
 */
#ifndef QKMLA_H
#define QKMLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
enum {
    QKMLA_OK = 0,
    QKMLA_ERR_INVALID = -1,       /* bad argument: null pointer, size, alignment */
    QKMLA_ERR_UNSUPPORTED = -2,   /* valid but not built (dtype / dims combination) */
    QKMLA_ERR_CUDA = -3,          /* a CUDA runtime/driver call failed */
    QKMLA_ERR_WORKSPACE = -4,     /* workspace missing or smaller than required */
    QKMLA_ERR_DEVICE_BOUNDS = -5, /* device saw a page id / length out of range */
    QKMLA_ERR_TIMEOUT = -6        /* device bounded wait expired */
};

/* Element types.  QKMLA_E4M3 names the 8-bit latent cache of qkmla_append_q8 and
 * qkmla_decode_ext; no other call takes it. */
enum { QKMLA_F32 = 0, QKMLA_BF16 = 1, QKMLA_E4M3 = 2 };

/* Flags. */
enum {
    /* Plain MLA (the comparator without QK normalisation): absorb writes
     * q~ = W^K_g q and alpha^q = 1; append stores the raw RoPE key and
     * alpha^k = 1; decode uses l = scale * (q~ . c_t + q_rope . k^rope_t). */
    QKMLA_FLAG_PLAIN_MLA = 1u,
    /* Decode: force the CUDA-core (SIMT) kernel even where the tensor-core
     * kernel applies.  Used to cross-check the two kernels. */
    QKMLA_FLAG_FORCE_SIMT = 2u,
    /* Decode, test hook for the failure path: the 64-row tensor-core kernel's
     * loader issues no tile from the second one on and every wait gives up
     * after 1 ms, so a call whose sequences span two or more tiles ends with
     * QKMLA_ERR_TIMEOUT in the status word (outputs undefined) and leaves the
     * context usable.  QKMLA_ERR_UNSUPPORTED for arguments that select another
     * kernel.  Never set outside tests. */
    QKMLA_FLAG_TEST_STALL = 4u,
    /* Append and decode: A^k_cache holds IEEE half-precision scalars
     * ([num_slots][G], 2 bytes each, round-to-nearest-even of the fp32
     * alpha^k) instead of fp32.  Halves the scalar cache, the method's only
     * storage overhead over MLA (Technical Summary, Key Contributions and
     * Results).  alpha^k = 1/sqrt(mean k^2 + eps) stays in fp16's normal range
     * (6.1e-5 .. 65504) for key RMS up to ~16000 and eps down to 2.3e-10; 11
     * significant bits keep each content logit within 2^-11 of its fp32 value.
     * Ignored with QKMLA_FLAG_PLAIN_MLA. */
    QKMLA_FLAG_ALPHA_F16 = 8u
};

/*
 * qkmla_absorb_query -- query side of the absorbed formulation.
 * Source: Technical Summary, Methodology, "Static Weight Absorption" (gamma_k
 * and gamma_q pre-multiply the query before the latent dot product) and the
 * decode-logit equation (alpha^q_{i,h} is the query's inverse RMS).
 *
 *   alpha_q[r][h]    = 1 / sqrt(mean_j q[r][h][j]^2 + eps)
 *   q_tilde[r][h][n] = sum_j W^K[g(h)][n][j] * q[r][h][j] * gamma_q[j] * gamma_k[j]
 *
 * q        [rows][H][d_h] fp32          gamma_q, gamma_k [d_h] fp32
 * w_k      [G][d_c][d_h]  fp32 (k_{t,g} = c_t W^K_g, i.e. W^K_g is d_c x d_h)
 * q_tilde  [rows][H][d_c] in qt_dtype (QKMLA_F32 or QKMLA_BF16, RNE cast)
 * alpha_q  [rows][H] fp32
 * PLAIN_MLA: gamma_* are ignored (may be NULL), alpha_q = 1.
 * Errors: INVALID for null pointers or non-positive sizes, H % G != 0,
 * d_h > 256 or d_c % 8 != 0; UNSUPPORTED for another qt_dtype.
 */
int qkmla_absorb_query(const float* q, const float* gamma_q, const float* gamma_k,
                       const float* w_k, int rows, int H, int G, int d_h, int d_c,
                       float eps, unsigned flags, void* q_tilde, int qt_dtype,
                       float* alpha_q, void* stream);

/*
 * qkmla_append -- write new tokens into the latent cache and A^k_cache.
 * Source: Technical Summary, Methodology, "Dynamic Scalar Caching" (one
 * inverse-RMS scalar per token and KV group), "Cache Layout" (keep c_t, add
 * the scalar cache, never store full keys) and "Blockwise Normalization"
 * (the RoPE part is normalised separately, as a materialised vector).
 *
 * For each new token n with slot s = slot_mapping[n] (s < 0: skipped):
 *   kv[s][0:d_c]   = cast(c_new[n])                       (bit-exact RNE cast)
 *   ak[s][g]       = 1 / sqrt(mean_j (c^ W^K_g)_j^2 + eps)  with c^ the stored latent
 *   kv[s][d_c:]    = cast(k_rope_new[n] * gamma_rope_k * beta_n),
 *                    beta_n = 1 / sqrt(mean_j k_rope_new[n][j]^2 + eps)
 * c_new [N][d_c] fp32, k_rope_new [N][d_r] fp32 (post-RoPE), w_k as above,
 * gamma_rope_k [d_r] fp32 or NULL (ones), slot_mapping [N] int64 device.
 * kv_cache [num_slots][d_c+d_r] in cache_dtype, ak_cache [num_slots][G] fp32
 * (fp16, the RNE cast of the fp32 value, with QKMLA_FLAG_ALPHA_F16).
 * PLAIN_MLA: the raw RoPE key is stored and ak = 1.
 * A slot >= num_slots is a device-side bounds error (skipped, status set).
 * N == 0 is a no-op.  Errors: INVALID / UNSUPPORTED as for absorb; d_h <= 256.
 */
int qkmla_append(const float* c_new, const float* k_rope_new, const float* w_k,
                 const float* gamma_rope_k, const int64_t* slot_mapping, int N, int G,
                 int d_c, int d_h, int d_r, float eps, unsigned flags, void* kv_cache,
                 int cache_dtype, void* ak_cache, int64_t num_slots, void* stream);

/*
 * qkmla_append_rope -- qkmla_append for RoPE keys that are not yet rotated:
 * each new token's RoPE key is first rotated by its position, then normalised
 * and stored exactly as qkmla_append stores a post-RoPE key.
 * Source: as qkmla_append, and Technical Summary, Methodology, "Blockwise
 * Normalization" (the RoPE part is a materialised vector normalised on its
 * own; the normalised vector is the rotated one).
 *
 * Rotation (the original rotary formulation; the pages name none): interleaved
 * pairs (x_2i, x_2i+1) of the d_r-vector turn by positions[n] * rope_theta^(-2i/d_r).
 * Angles are reduced exactly enough for positions up to 2^24 (fp64 frequency,
 * error-free fp32 product, two-part 2*pi reduction).
 * k_rope_raw [N][d_r] fp32 (before rotation); positions [N] int32 device.
 * Errors: as qkmla_append, and INVALID for a missing positions array, d_r odd
 * or rope_theta <= 1; UNSUPPORTED for d_r > 64.
 */
int qkmla_append_rope(const float* c_new, const float* k_rope_raw, const int32_t* positions, float rope_theta,
                      const float* w_k, const float* gamma_rope_k, const int64_t* slot_mapping, int N, int G,
                      int d_c, int d_h, int d_r, float eps, unsigned flags, void* kv_cache, int cache_dtype,
                      void* ak_cache, int64_t num_slots, void* stream);

/*
 * qkmla_append_q8 -- write new tokens into the 8-bit latent cache.
 *
 * The cache of the pages' method (latent, alpha^k, RoPE key) with the latent in
 * e4m3 (4 exponent, 3 mantissa bits, largest value 448) and one fp32 scale a
 * token.  The latent is the cache's only "head", and a scale covers one token:
 * outlier tokens (tens of times the others) would otherwise take the codes of
 * their neighbours.  Scales are powers of two, so code x scale is exact.
 *
 * For each new token n with slot s = slot_mapping[n] (s < 0: skipped):
 *   kv_scale[s]    = 2^e, the least with max_j |c_new[n][j]| <= 448 2^e (at least
 *                    2^-126); 0 for an all-zero latent
 *   kv[s][0:d_c]   = e4m3(c_new[n] / kv_scale[s]), round to nearest even; a value
 *                    that is not finite is stored as NaN
 *   ak[s][g]       = 1 / sqrt(mean_j (c^ W^K_g)_j^2 + eps)  with c^ the stored
 *                    latent (code x scale)
 *   kv[s][d_c:]    = bf16(RoPE key, rotated by positions[n] if positions is given,
 *                    normalised) as qkmla_append / qkmla_append_rope store it
 * kv_cache [num_slots][d_c + 2 d_r] bytes: d_c codes, then d_r bf16 values.
 * kv_scale [num_slots] fp32.  ak_cache as in qkmla_append.  positions [N] int32
 * or NULL (k_rope_new is already rotated; rope_theta is then ignored).
 * PLAIN_MLA: the raw RoPE key is stored and ak = 1.
 * A slot >= num_slots is a device-side bounds error (skipped, status set).
 * N == 0 is a no-op.  Errors: INVALID for null pointers, sizes, odd d_c, d_h >
 * 256, misaligned bases; UNSUPPORTED for d_c > 512 or d_r > 64.
 */
int qkmla_append_q8(const float* c_new, const float* k_rope_new, const int32_t* positions, float rope_theta,
                    const float* w_k, const float* gamma_rope_k, const int64_t* slot_mapping, int N, int G, int d_c,
                    int d_h, int d_r, float eps, unsigned flags, void* kv_cache, float* kv_scale, void* ak_cache,
                    int64_t num_slots, void* stream);

/*
 * qkmla_project_query -- the query projection ahead of qkmla_absorb_query,
 * with the RoPE rotation of the RoPE block fused in.
 * Source: thelatestinai.com abstract (the static key weight is absorbed into
 * the MLA query-side projection: the query comes from the layer input through
 * W^Q, then qkmla_absorb_query folds gamma_q * gamma_k and W^K_g into it);
 * Technical Summary, Methodology, "Blockwise Normalization".
 *
 *   [q_h | r_h] = x W^Q_h^T,  q[r][h] = q_h,  q_rope[r][h] = RoPE(r_h, positions[r])
 *
 * x [rows][d_x] bf16; w_q [H][d_h + d_r][d_x] bf16 (row j of W^Q_h holds output
 * j's weights: the d_h content outputs, then the d_r RoPE outputs);
 * positions [rows] int32 device (RoPE position of each query row);
 * q [rows][H][d_h] fp32 (qkmla_absorb_query's input); q_rope [rows][H][d_r]
 * fp32, rotated as in qkmla_append_rope, not normalised (qkmla_decode's input).
 * Tensor cores, fp32 accumulation.  Errors: INVALID for null pointers, bad
 * sizes or alignment, rope_theta <= 1 with d_r > 0; UNSUPPORTED for d_x % 64,
 * odd d_h or d_r, d_r > 64, or d_h + d_r not in {96, 128, 160, 192, 256}.
 */
int qkmla_project_query(const void* x, const void* w_q, const int32_t* positions, float rope_theta, int rows,
                        int d_x, int H, int d_h, int d_r, float* q, float* q_rope, void* stream);

/* Arguments of qkmla_decode (plain pointers and sizes). */
typedef struct qkmla_decode_args {
    const void* q_tilde;        /* [B][s_q][H][d_c] in cache_dtype (from absorb); bf16 with QKMLA_E4M3 */
    const float* alpha_q;       /* [B][s_q][H] fp32 */
    const float* q_rope;        /* [B][s_q][H][d_r] fp32, post-RoPE, not normalised */
    const float* gamma_rope_q;  /* [d_r] fp32 or NULL (ones) */
    const void* kv_cache;       /* [num_slots][d_c+d_r] cache_dtype; with QKMLA_E4M3 rows of d_c codes and d_r bf16 */
    const void* ak_cache;       /* [num_slots][G] fp32 (fp16 with QKMLA_FLAG_ALPHA_F16) */
    const int32_t* seq_lens;    /* [B] int32 device: tokens in the cache incl. this step's s_q */
    const int32_t* page_table;  /* [B][max_pages] int32 device, or NULL (contiguous) */
    int64_t num_slots;          /* slots in kv_cache / ak_cache (multiple of page_size) */
    int page_size;              /* tokens per page (> 0) */
    int max_pages;              /* page-table row length; max tokens = max_pages*page_size, below 2^31 - 4096 */
    int B, s_q, H, G, d_c, d_r;
    int cache_dtype;            /* QKMLA_F32 or QKMLA_BF16; QKMLA_E4M3 in qkmla_decode_ext alone */
    float softmax_scale;        /* multiplies the whole logit, e.g. 1/sqrt(d_h+d_r) */
    float eps;                  /* RMS epsilon of the RoPE query normalisation */
    unsigned flags;             /* QKMLA_FLAG_* */
    int num_splits;             /* 0: automatic; k >= 1 (to 1024): k equal token ranges per sequence; with k > 256
                                 * or B k > 65535 the CUDA-core kernel serves the call */
    void* workspace;            /* device scratch, >= qkmla_decode_workspace_size(args) bytes */
    size_t workspace_bytes;
    void* o;                    /* [B][s_q][H][d_c] output in o_dtype */
    int o_dtype;                /* QKMLA_F32 or QKMLA_BF16 */
    float* lse;                 /* [B][s_q][H] fp32: natural log of sum_t exp(l_t); may be NULL */
} qkmla_decode_args;

/*
 * qkmla_decode_workspace_size -- bytes of device scratch qkmla_decode needs
 * for these arguments (split-KV partial outputs and scheduler metadata).  Only
 * the shape fields, flags, cache_dtype and num_splits are read.  Returns 0 for
 * arguments qkmla_decode would reject.  Depends on the current device.
 */
size_t qkmla_decode_workspace_size(const qkmla_decode_args* a);

/*
 * qkmla_decode -- QK-Normed MLA decode attention over the latent cache.
 * Source: Technical Summary, Methodology, decode-logit equation (row scaling
 * by alpha^q, column scaling by alpha^k, before the softmax) and "Blockwise
 * Normalization" (the RoPE logit uses materialised normalised vectors); the
 * abstract's "preserves MLA's latent decode path" (values are the latents).
 *
 * Query i of sequence b attends to tokens t < seq_lens[b] - s_q + i + 1.
 * q^rope = q_rope * gamma_rope_q / sqrt(mean(q_rope^2) + eps) per head.
 * o[b][i][h] = sum_t p_t c_t with p = softmax_t(l); lse = log sum_t exp(l_t).
 * Long contexts are split over CTAs (split-KV) and merged by a combine kernel.
 * Errors: INVALID (null pointer, bad dims, H % G, d_c % 64 for bf16, ...),
 * UNSUPPORTED (heads per group H / G other than 1, 2, 4, 8 or 16; d_c > 512
 * or d_r > 128; a cache or output dtype other than fp32 / bf16), WORKSPACE
 * (workspace smaller than required).  Device-side:
 * seq_len < s_q or > max_pages*page_size, or a page id outside
 * [0, num_slots/page_size), set QKMLA_ERR_DEVICE_BOUNDS; the sequence's
 * affected rows are then undefined.
 */
int qkmla_decode(const qkmla_decode_args* a, void* stream);

/* What qkmla_decode_ext takes besides qkmla_decode_args. */
typedef struct qkmla_decode_ext_args {
    const float* kv_scale;      /* [num_slots] fp32, with cache_dtype QKMLA_E4M3 only (else NULL) */
    int window;                 /* 0: every token; w >= 1: the last w tokens of each query */
    int sinks;                  /* with a window: the first tokens that stay visible */
} qkmla_decode_ext_args;

/*
 * qkmla_decode_ext -- qkmla_decode over an 8-bit cache, through a sliding window
 * with sinks, or both.
 *
 * 8-bit cache (cache_dtype QKMLA_E4M3): kv_cache and kv_scale as
 * qkmla_append_q8 writes them; q_tilde is bf16.  The stored latent is
 * c^_t = kv_scale_t x codes_t, in the logits and in the output; everything else
 * is qkmla_decode's definition.
 *
 * Window w, sinks f: query i of sequence b, of causal length n = seq_lens[b] -
 * s_q + i + 1, attends to the tokens t < n with t < f or t >= n - w.  What is
 * stored for tokens that a query does not see (NaN included) does not reach its
 * result, and pages that no query of the step sees are not read; a tile of up to 64
 * tokens that holds a visible one is loaded whole, so its page-table entry has
 * to be valid.
 *
 * With an 8-bit cache or a window, seq_lens[b] may be anything from 0 to
 * max_pages * page_size: a query without a visible token (an idle batch slot)
 * gives o = 0 and lse = -inf.  With neither, the call is qkmla_decode.  A NaN in
 * what a query sees, or in its own row, is NaN in all of its o and lse.
 *
 * Accuracy: fp32 sums, with the output's weights rounded -- 8-bit cache: p_t
 * kv_scale_t to two 8-bit parts, off by 2^-8 of itself (2^-11 more from fp16); one
 * below 2^-7 of the row's largest instead by up to 2^-14 of that largest (2^-15, 2^-16,
 * 2^-19 in ranges of more than 2^11, 2^13, 2^14 tokens), up or down in proportion by
 * the token's place, so that N of them are off by sqrt(N) such steps together and not
 * by N; bf16 cache: as qkmla_decode.  Tensor-core kernels serve the
 * 8-bit cache for (d_c, d_r) of (512, 64), (256, 32 or 64) and (128, 32 or 64), H a
 * multiple of 16, G <= 8, B <= 4096, page sizes 16, 32 or a multiple of 64 and
 * 16-byte aligned bases, and windows over the bf16 cache where qkmla_decode has one;
 * the CUDA-core kernel serves the rest.
 *
 * The workspace size, the kernel's name and the launches come from the _ext
 * forms of their calls.  Errors: as qkmla_decode, and INVALID for a null
 * argument block, a negative window or sinks, sinks without a window, kv_scale
 * without QKMLA_E4M3 or the reverse, or an odd d_c with QKMLA_E4M3.
 */
int qkmla_decode_ext(const qkmla_decode_args* a, const qkmla_decode_ext_args* e, void* stream);
size_t qkmla_decode_ext_workspace_size(const qkmla_decode_args* a, const qkmla_decode_ext_args* e);
const char* qkmla_decode_ext_kernel_name(const qkmla_decode_args* a, const qkmla_decode_ext_args* e);
int qkmla_decode_ext_launch_count(const qkmla_decode_args* a, const qkmla_decode_ext_args* e);

/*
 * qkmla_get_device_status -- synchronise `stream`, return and clear the
 * current device's status word (QKMLA_OK or the first device-side error since
 * the last call).  Returns QKMLA_ERR_CUDA if synchronisation fails.
 */
int qkmla_get_device_status(void* stream);

/* Human-readable name of a return code (static string). */
const char* qkmla_status_string(int status);

/* Library version: major*10000 + minor*100 + patch. */
int qkmla_version(void);

/*
 * qkmla_decode_kernel_name -- which decode kernel qkmla_decode would launch for
 * these arguments on the current device: "tcgen05" (tensor-core kernel),
 * "simt" (CUDA-core kernel) or "invalid".  Static string.
 */
const char* qkmla_decode_kernel_name(const qkmla_decode_args* a);

/*
 * qkmla_decode_launch_count -- number of kernels one qkmla_decode call with
 * these arguments launches on the stream (tensor-core path: decode and
 * combine, plus a split-scheduler kernel ahead of them for batches of more
 * than 128 sequences -- smaller batches are planned inside the decode and
 * combine kernels; CUDA-core path: decode, plus combine when it splits).
 * Returns 0 for arguments qkmla_decode would reject.
 */
int qkmla_decode_launch_count(const qkmla_decode_args* a);

/*
 * qkmla_decode_noalloc -- qkmla_decode for callers that cannot allocate
 * device memory when they decode: a runtime that hands out only pre-planned
 * buffers, a plugin whose host owns every allocation, or a thread that must
 * not enter the CUDA allocator.  The paper has no counterpart to this call.
 *
 * Same arguments and results as qkmla_decode, except that `workspace` and
 * `workspace_bytes` are ignored: the split-KV partials and scheduler data live
 * in a fixed array of qkmla_decode_noalloc_max_workspace() bytes (64 MiB)
 * inside the library.  The array is part of the library's device code, so it
 * is reserved on a GPU when that code is loaded there -- with CUDA's default
 * lazy loading, at the first launch of any of the library's kernels on that
 * device; with CUDA_MODULE_LOADING=EAGER, when a context is created -- and is
 * held until the process exits.  The call allocates nothing.  Arguments
 * needing more scratch than that return QKMLA_ERR_WORKSPACE before anything is
 * launched.
 * The first call on a device resolves the array's address on that device (it
 * must be current) and keeps it for the process; make that first call before
 * any stream capture, and do not use the library across a cudaDeviceReset
 * (the kept address would be stale).  All calls on a device share the array:
 * calls whose kernels can overlap on the GPU (different streams with no
 * ordering between them) race on it.  The array keeps the previous call's
 * contents; decode writes every scratch entry it reads, so nothing needs to
 * start at zero.
 */
int qkmla_decode_noalloc(const qkmla_decode_args* a, void* stream);

/*
 * qkmla_up_project -- per-head values from the latent-space decode output.
 * Source: Technical Summary, Problem Statement (MLA keeps the low-dimensional
 * latent and recovers per-head quantities through up-projections, as W^K_g
 * recovers the key); the abstract (decode keeps the latent path, so attention
 * returns o = sum_t p_t c_t).  The value of head h is recovered once per query
 * row instead of once per cached token:
 *
 *   out[r][h][j] = sum_n o[r][h][n] * W^V[g(h)][n][j],   g(h) = h / (H / G_v)
 *
 * which equals softmax attention over materialised values c_t W^V_{g(h)}
 * (the softmax weights sum to one).
 * o     [rows][H][d_c] in o_dtype (QKMLA_F32 or QKMLA_BF16): qkmla_decode's output
 * w_v   [G_v][d_c][d_v] bf16 (G_v = H: one matrix per head)
 * out   [rows][H][d_v] in out_dtype (QKMLA_F32 or QKMLA_BF16)
 * Tensor cores, fp32 accumulation; an fp32 o is split into two bf16 parts
 * (fp32-level accuracy).  Errors: INVALID for null pointers, non-positive
 * sizes, H % G_v != 0 or a base not 16-byte aligned; UNSUPPORTED for other
 * dtypes, d_c % 64 != 0, or d_v not in {64, 128, 192, 256}.
 */
int qkmla_up_project(const void* o, int o_dtype, const void* w_v, int rows, int H, int G_v, int d_c,
                     int d_v, void* out, int out_dtype, void* stream);

/* Layouts and frequencies of qkmla_rope. */
enum { QKMLA_ROPE_INTERLEAVED = 0, QKMLA_ROPE_HALVES = 1 };
enum { QKMLA_ROPE_PLAIN = 0, QKMLA_ROPE_LINEAR = 1, QKMLA_ROPE_YARN = 2, QKMLA_ROPE_GIVEN = 3 };

/* Arguments of qkmla_rope. */
typedef struct qkmla_rope_args {
    const void* x;              /* element (r, h, j) at x + r x_row_stride + h x_head_stride + j, in dtype */
    void* out;                  /* likewise; may be x with x's strides (in place), else no overlap with x */
    const int32_t* positions;   /* [rows] int32 device: any value */
    int64_t x_row_stride, x_head_stride, out_row_stride, out_head_stride;   /* in elements */
    int rows, heads, d_r;       /* d_r even, at most 256: the elements of each head that are rotated */
    int dtype;                  /* QKMLA_F32 or QKMLA_BF16, of x and out */
    int layout;                 /* pairs (2i, 2i + 1), or with QKMLA_ROPE_HALVES (i, i + d_r / 2) */
    int inverse;                /* not 0: turned back, by the opposite angles (also the backward pass) */
    int scaling;                /* QKMLA_ROPE_*: how the pairs' frequencies are formed */
    float theta;                /* frequency of pair i: theta^(-2i/d_r); > 1 (not read with GIVEN) */
    float factor;               /* LINEAR, YARN: how many times the original context */
    int original_context;       /* YARN: tokens of the original context */
    float beta_fast, beta_slow; /* YARN: turns within it, usually 32 and 1 */
    float attention_factor;     /* multiplies the result; 0 means 1 */
    const double* frequencies;  /* GIVEN: HOST array [d_r / 2], radians a position; read during the call */
} qkmla_rope_args;

/*
 * qkmla_rope -- rotary positions on RoPE blocks that lie on their own or inside a
 * head: queries and keys whose positions are scaled for a long context or whose
 * pairs are halves apart, which the rotations fused into qkmla_project_query and
 * qkmla_append_rope (interleaved, unscaled) do not serve.
 *
 *   (a, b) -> attention_factor (a cos - b sin, a sin + b cos),  angle = positions[r] f_i
 *
 * f_i = theta^(-2i/d_r); LINEAR: divided by factor; YARN: with u_i the ramp from 0 at
 * pair floor(c(beta_fast)) to 1 at pair ceil(c(beta_slow)), both within [0, d_r - 1],
 * c(n) = d_r ln(original_context / (2 pi n)) / (2 ln theta): f_i (u_i / factor + 1 - u_i);
 * GIVEN: frequencies[i].  Elements outside the rotated part are neither read nor
 * written.  Computed in fp32, one rounding to bf16.  A frequency is a 64-bit number, to 2^-48 of
 * itself (2^-46 on YARN's ramp; theta up to 10^8): an angle of N turns, N = |positions[r] f_i| /
 * (2 pi), is off by at most N times that and 2^-26 of a turn, 2^-25 for positions below 2^24 and
 * f_i <= 1 off the ramp.
 * rows == 0 is a no-op.
 * Errors: INVALID for null pointers, sizes, an odd d_r, outputs that share elements (a stride
 * below d_r), unknown layout or scaling, theta <= 1, factor <= 0, bad betas, a frequency that is
 * not finite, misaligned elements; UNSUPPORTED for another dtype, d_r > 256 or more heads than a launch takes.
 */
int qkmla_rope(const qkmla_rope_args* a, void* stream);

/* Arguments of qkmla_read_cache. */
typedef struct qkmla_read_cache_args {
    const void* kv_cache;       /* [num_slots][d_c+d_r] cache_dtype; with QKMLA_E4M3 rows of d_c codes and d_r bf16 */
    const float* kv_scale;      /* [num_slots] fp32, with QKMLA_E4M3 only (else NULL) */
    const void* ak_cache;       /* [num_slots][G] fp32 (fp16 with QKMLA_FLAG_ALPHA_F16); NULL without ak */
    const int32_t* out_start;   /* [B+1] int32 device, not decreasing: output rows of each sequence */
    const int32_t* first;       /* [B] int32 device: a sequence's first token to be read, or NULL (0) */
    const int32_t* page_table;  /* [B][max_pages] int32 device, or NULL (contiguous) */
    int64_t num_slots;
    int page_size, max_pages;
    int B, rows, G, d_c, d_r;   /* rows: of the outputs; those outside [out_start[0], out_start[B]) stay as they are */
    int cache_dtype;            /* QKMLA_F32, QKMLA_BF16 or QKMLA_E4M3 */
    int out_dtype;              /* QKMLA_F32 or QKMLA_BF16, of c and r */
    unsigned flags;             /* QKMLA_FLAG_ALPHA_F16 */
    void* c;                    /* [rows][d_c] the stored latents */
    void* r;                    /* [rows][d_r] the stored (normalised) RoPE keys */
    float* ak;                  /* [rows][G] fp32, or NULL */
} qkmla_read_cache_args;

/*
 * qkmla_read_cache -- the counterpart of qkmla_append and qkmla_append_q8: rows of
 * the cache, wherever their pages lie, as contiguous arrays (to move a prefix to
 * another cache, cache type or device, or to keep it).
 *
 * Row n, out_start[b] <= n < out_start[b+1], is token first[b] + n - out_start[b] of
 * sequence b: c = cast(c^_t) with c^_t the stored latent (8-bit cache: code x scale),
 * r = cast(k^rope_t), ak = alpha^k_t; casts to a narrower type round to nearest even.
 * A token outside [0, max_pages * page_size) or a page id outside [0, num_slots /
 * page_size) sets QKMLA_ERR_DEVICE_BOUNDS and leaves its row as it was.  rows == 0 is
 * a no-op.  Errors: INVALID for null pointers, sizes, misaligned elements, kv_scale
 * without QKMLA_E4M3 or the reverse, an odd d_c with QKMLA_E4M3; UNSUPPORTED for other
 * dtypes.
 */
int qkmla_read_cache(const qkmla_read_cache_args* a, void* stream);

/*
 * qkmla_prefill_pack_weights -- the up-projections in the layout qkmla_prefill's
 * tensor-core product reads: once for a layer's weights.
 * w_k [G][d_c][d_h] fp32, w_v [G_v][d_c][d_v] bf16 (as in qkmla_append and
 * qkmla_up_project); packed: qkmla_prefill_weights_size(...) bytes, 16-byte aligned.
 * Each matrix is stored as fp16 times a power of two of its own (its largest value in
 * [1, 2)): W^K is off by 2^-11 of itself, W^V exact, down to 2^-14 of the matrix's
 * largest value.
 * qkmla_prefill_weights_size: 0 for sizes qkmla_prefill does not serve.
 * Errors: INVALID for null pointers, sizes or misaligned bases; UNSUPPORTED for sizes
 * that qkmla_prefill does not serve.
 */
size_t qkmla_prefill_weights_size(int G, int G_v, int d_c, int d_h, int d_v);
int qkmla_prefill_pack_weights(const float* w_k, const void* w_v, int G, int G_v, int d_c, int d_h, int d_v,
                               void* packed, void* stream);

/* Arguments of qkmla_prefill. */
typedef struct qkmla_prefill_args {
    const void* q;              /* (row, h, j) at q + row q_row_stride + h q_head_stride + j, in q_dtype: not normalised */
    const void* q_rope;         /* likewise, post-RoPE, not normalised */
    int64_t q_row_stride, q_head_stride, qr_row_stride, qr_head_stride;   /* in elements, multiples of 4 */
    const float* gamma_q;       /* [d_h] */
    const float* gamma_k;       /* [d_h] */
    const float* gamma_rope_q;  /* [d_r] or NULL (ones) */
    const void* weights;        /* from qkmla_prefill_pack_weights */
    const void* kv_cache;       /* as in qkmla_decode_args: QKMLA_BF16, or QKMLA_E4M3 with kv_scale */
    const float* kv_scale;      /* [num_slots] fp32 with QKMLA_E4M3, else NULL */
    const void* ak_cache;       /* [num_slots][G] fp32 (fp16 with QKMLA_FLAG_ALPHA_F16) */
    const int32_t* chunk_start; /* [B+1] int32 device, chunk_start[0] = 0, not decreasing, the last <= rows */
    const int32_t* seq_lens;    /* [B] int32 device: tokens in the cache incl. the chunk's */
    const int32_t* page_table;  /* [B][max_pages] int32 device, or NULL (contiguous) */
    int64_t num_slots;
    int64_t total_tokens;       /* at least the sum of seq_lens: sizes the workspace */
    int page_size, max_pages;
    int B, rows, H, G, G_v, d_c, d_h, d_r, d_v;
    int cache_dtype, q_dtype, o_dtype;   /* q_dtype, o_dtype: QKMLA_F32 or QKMLA_BF16 */
    float softmax_scale, eps;
    int window, sinks;          /* as in qkmla_decode_ext_args */
    unsigned flags;             /* QKMLA_FLAG_ALPHA_F16 */
    void* workspace;            /* device scratch, >= qkmla_prefill_workspace_size(args) bytes, 256-byte aligned */
    size_t workspace_bytes;
    void* o;                    /* [rows][H][d_v] in o_dtype: per-head values */
    float* lse;                 /* [rows][H] fp32, or NULL */
} qkmla_prefill_args;

/*
 * qkmla_prefill -- attention of a chunk of new tokens over the paged latent cache,
 * the chunk's own tokens (already appended) among it: a prompt's prefill whole or in
 * chunks, several sequences a call, single decode tokens among them.
 * Source: as qkmla_decode; Technical Summary, Problem Statement (keys and values are
 * up-projections of the latent).  With many query rows a token it costs less to recover
 * each cached token's key and value once, k_{t,g} = alpha^k_{t,g} c^_t W^K_g and
 * v_t = c^_t W^V, than to attend in latent space: 2 (d_h + d_r + d_v) flops a pair and
 * head instead of 2 (2 d_c + d_r).  The cache, its bytes and the result are the same.
 *
 * Row r of sequence b, chunk_start[b] <= r < chunk_start[b+1], is query i = r - chunk_start[b]
 * of n_b: it attends to tokens t < n = seq_lens[b] - n_b + i + 1, with a window w and sinks f
 * to those with t < f or t >= n - w;
 *   l = softmax_scale ( q^ . k_{t,g(h)} + q^rope . k^rope_t ),  q^ = q gamma_q gamma_k / rms(q),
 *   q^rope = q_rope gamma_rope_q / rms(q_rope),  rms(z) = sqrt(mean z^2 + eps)
 *   o[r][h] = sum_t softmax_t(l) v_t,  lse = ln sum_t exp(l_t)
 * = qkmla_absorb_query, qkmla_decode_ext and qkmla_up_project over the same cache.
 * A query without a visible token gives o = 0, lse = -inf.  Rows from chunk_start[B] on
 * stay as they are.  Stored values that no query of a row's step sees do not reach its
 * result, NaN included, and pages of such tokens alone are not looked up; a NaN in what a
 * query sees, or in its own row, is NaN in its o and lse.
 *
 * For few rows a sequence decode costs less (absorb + decode + up-projection against this call,
 * 16 sequences of 4096 tokens: 128 heads, d_c 512, one row 96 against 237 us, equal between 8 and
 * 12 rows; 16 heads, d_c 256, one row 26 against 80, equal at about 32).
 *
 * Accuracy: fp16 operands (11 significant bits) of tensor-core products, fp32 sums:
 * recovered keys and values, normalised queries (the gains times one power of two a call) and
 * softmax weights are each off by 2^-11 of themselves, values of less than 2^-13 of the largest
 * among 128 neighbouring tokens by up to 2^-25 of that largest; where 128 neighbouring
 * tokens' latents (of those that some row of the step sees, zeros left out) differ by more
 * than 2^12, or leave 2^-40 .. 2^40, their values and weights are bf16 (2^-8).  With l the
 * smallest of those 128 latents' sizes, a weight p loses bits where p l is below 2^-21 of the row's
 * largest p l, and may be 0 below 2^-32 of it.  RoPE keys are taken as fp16: up to 65504.
 *
 * Sizes: d_h and d_v 64 or 128, d_r 32 or 64, d_c a multiple of 64 up to 512, H / max(G, G_v)
 * 1, 2, 4, ... or 128, the larger of G and G_v a multiple of the other, B <= 4096, any page size; 16-byte
 * aligned bases (o: 32-byte).
 * Device-side: a seq_len outside [0, max_pages * page_size], lengths that add up to more than
 * total_tokens, chunk starts out of order or beyond rows, or a page id outside [0, num_slots /
 * page_size) set QKMLA_ERR_DEVICE_BOUNDS; the affected sequences' rows are then undefined (with
 * chunk starts out of order, every row).
 * rows == 0 is a no-op.  Errors: INVALID for null pointers, sizes, strides, alignment, window or
 * sinks as in qkmla_decode_ext, kv_scale without QKMLA_E4M3 or the reverse; UNSUPPORTED for other
 * sizes or dtypes, or with QKMLA_FLAG_PLAIN_MLA; WORKSPACE.
 * qkmla_prefill_workspace_size: 0 for arguments that the call rejects; reads the sizes alone.  Depends
 * on the current device.  Keys and values of all tokens lie there at once: 2 (G d_h + G_v d_v + 64)
 * bytes a token of total_tokens, rounded up to 128 tokens a sequence (8 groups of 128 + 128: 4.2 KB).
 */
int qkmla_prefill(const qkmla_prefill_args* a, void* stream);
size_t qkmla_prefill_workspace_size(const qkmla_prefill_args* a);

/* Bytes of scratch qkmla_decode_noalloc can use (its fixed array). */
size_t qkmla_decode_noalloc_max_workspace(void);

#ifdef __cplusplus
}
#endif

#endif /* QKMLA_H */
