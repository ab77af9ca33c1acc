/* clsample.h: C ABI of the GB300 (sm_103a) batched constrained logits sampler.
 *
 * One call turns a [B, V] next-token logits matrix into one token id per row, plus the
 * drawn token's logprob.  For every row it applies, in order:
 *
 *   1. sanitising of non-finite logits
 *        (SGLang source teardown (10): Sampling, Grammar and structured output,
 *         section "_preprocess_logits");
 *   2. frequency / presence penalties (additive), then the repetition penalty (scaling),
 *      then sparse logit_bias (a repeated id keeps its last value)
 *        (same page, sections "Order semantics of the penalties" and "Why logit_bias is
 *         built from triples");
 *   3. the int32 grammar bitmask: bit (i & 31) of word i >> 5 equal to 0 sets logit i to
 *      -inf, before any truncation
 *        (same page, section "Bitmask: one int32 covers 32 tokens");
 *   4. the greedy rule: temperature < 1e-5 (GLM-5.3 inference (7): output side, section
 *      "Sampling") or top_k in {0, 1} (SGLang page, section "Field groups");
 *   5. temperature, then top-k -> top-p -> min-p truncation on the tempered distribution
 *        (SGLang page, section "The maths of the three cuts": S_k, S_p, S_m);
 *   6. an exponential race keyed by (seed, position): token = argmax_i p_i / E_i over the
 *      kept set, E_i = -ln U_i with U_i from Philox4x32-10 (Salmon et al., SC'11) at
 *      counter (i / 4, position, 0) and key seed, so a request's draw does not depend on
 *      the batch it is in (SGLang page, section "Call site"; GLM-5.3 page: one random
 *      stream per request);
 *   7. the logprob of the drawn token under the full tempered distribution, computed as
 *      log-softmax (SGLang page, section "Numerical consistency of logprobs").
 *
 * Threading and ownership.  A handle is bound to the CUDA device that was current at
 * clsample_create and owns device scratch sized for max_batch rows (row order and
 * counters, per-slice records, per-row lists of penalised and biased tokens, compacted
 * candidates, and a spill area of one row per batch row; about 1.5 MB per row for
 * V = 151936).  Every array in clsample_args_t is a DEVICE pointer owned by the caller;
 * it must stay valid until the work enqueued on the stream has finished.  The logits are
 * read-only (never written in place).  Calls on one handle must be ordered (one stream,
 * or streams joined by events): they share the handle's scratch.  Separate handles are
 * independent.
 *
 * Errors.  Every entry point validates its arguments on the host, without any device
 * synchronisation, and returns a negative CLSAMPLE_ERR_* code on a bad argument;
 * nothing is enqueued then.  Data errors found on the device (ids outside [0, V),
 * decreasing CSR offsets, NaN parameters, a row with no allowed token) never trap:
 * they go to the per-row status (OK < OVERFLOW < INVALID, ordered by severity so that
 * a MAX reduction over rows gives one verdict; SGLang page, section
 * "LogitsProcessorOutput"), and such a row gets token -1 and logprob -inf.
 */
#ifndef CLSAMPLE_H
#define CLSAMPLE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* clsample_stream_t;
typedef struct clsample_handle clsample_t;

enum {
  CLSAMPLE_LOGITS_F32 = 0,  /* float32 logits */
  CLSAMPLE_LOGITS_BF16 = 1  /* bfloat16 logits, widened exactly to float32 */
};

/* Per-row status codes written to row_status. */
enum { CLSAMPLE_ROW_OK = 0, CLSAMPLE_ROW_OVERFLOW = 1, CLSAMPLE_ROW_INVALID = 2 };

/* Return codes. */
enum {
  CLSAMPLE_SUCCESS = 0,
  CLSAMPLE_ERR_NULL = -1,       /* a required pointer is NULL */
  CLSAMPLE_ERR_BATCH = -2,      /* B < 0 or B > max_batch */
  CLSAMPLE_ERR_VOCAB = -3,      /* V <= 0, V != the handle's vocab, or V > 262144 */
  CLSAMPLE_ERR_STRIDE = -4,     /* logits_row_stride < V or bitmask_row_stride < ceil(V/32) */
  CLSAMPLE_ERR_DTYPE = -5,      /* logits_dtype is not a CLSAMPLE_LOGITS_* value */
  CLSAMPLE_ERR_CUDA = -6,       /* a CUDA runtime call failed (launch, attribute, device) */
  CLSAMPLE_ERR_DEVICE = -7,     /* the current device is not the handle's or not sm_103 */
  CLSAMPLE_ERR_MODE = -8,       /* mode has a bit that is not a CLSAMPLE_MODE_* flag */
  CLSAMPLE_ERR_SHAPE = -9,      /* a count, head layout, head size or page size out of range */
  CLSAMPLE_ERR_ALIGN = -10      /* an address or stride that a kernel needs aligned is not */
};

/* Bits of clsample_args_t.mode (0: sequential truncation, one draw per row). */
enum {
  /* Top-p over the whole distribution, intersected with the top-k set (SGLang page,
   * the sampler's "joint" filter order), instead of top-p over the renormalised top-k
   * set.  Rows with a top-k cut and top_p < 1 then take the co-resident row-group route. */
  CLSAMPLE_MODE_JOINT_TOPK_TOPP = 1,
  /* Scoring only (SGLang page, logprobs-only computation): the same transforms, no draw.
   * Every row takes the greedy route whatever its parameters -- token = argmax of z',
   * logprobs at T_eff -- and the requested ids (tid_*) get their logprobs. */
  CLSAMPLE_MODE_SCORE_ONLY = 2,
  /* Batch fast path (SGLang page, "Field groups": the host-side batch booleans
   * is_all_greedy and need_top_k/top_p/min_p_sampling, and the sampler's simple-sampling
   * branch; GLM page, "Sampling").  The caller asserts that every row is greedy (T < 1e-5,
   * top_k 0 or 1, or SCORE_ONLY) or untruncated (top_p 1, min_p 0, top_k -1 or at least
   * the row's allowed tokens).  The call is then one sweep over the logits -- no
   * preparation launch -- with the same results as without the flag.  A row that breaks
   * the assertion, or has 2^20 or more history ids or 4095 or more bias entries, gets
   * status INVALID.  Requested-id and top-N logprobs are not available (ERR_MODE).
   * An untruncated row draws from candidates within 2e-3 of each slice's best fast race
   * score; a slice with more than 64 of them (not seen in practice) makes the row
   * OVERFLOW. */
  CLSAMPLE_MODE_FAST_SWEEP = 4
};

/* Arguments of one sampler call.  B rows, V vocabulary entries.
 *
 * mode              CLSAMPLE_MODE_* bits, 0 for plain sampling; other bits: ERR_MODE.
 * logits            [B, logits_row_stride] elements of logits_dtype, row-major.
 * temperatures      f32[B]; NULL = 1.0.  T < 1e-5 (including 0 and negatives) is greedy;
 *                   NaN or +inf is INVALID.
 * top_ks            i32[B]; NULL = -1.  -1 (or >= the number of allowed tokens) keeps the
 *                   whole vocabulary; 0 and 1 are greedy; < -1 is INVALID.  Every token
 *                   tied with the k-th largest probability is kept.
 * top_ps            f32[B]; NULL = 1.0.  Must lie in (0, 1], else INVALID.
 * min_ps            f32[B]; NULL = 0.0.  Must lie in [0, 1], else INVALID.
 * rep, freq, pres   f32[B] each, NULL = 1.0 / 0.0 / 0.0.  For a token seen c > 0 times in
 *                   the row's history: z -= freq*c; z -= pres; then z = z > 0 ? z/rep :
 *                   z*rep.  rep must be finite and > 0, freq and pres finite.
 * hist_offs/ids     CSR of the rows' token histories: ids hist_ids[hist_offs[r] ..
 *                   hist_offs[r+1]), duplicates counted.  NULL offs = no penalties.
 * bias_offs/ids/vals CSR of logit_bias entries; z += val; for a repeated id the LAST
 *                   entry of the row wins.  NULL offs = no bias.  NaN values are INVALID.
 * bitmask           i32[B, bitmask_row_stride] words, bit i & 31 of word i >> 5 allows
 *                   token i; NULL = unconstrained.  A row of all -1 words is unconstrained.
 * seeds             u64[B]; NULL = 0 for every row.  The request's random key.
 * positions         i64[B]; NULL = `step` for every row.  The request's token position;
 *                   rows of one request at different positions draw independently.
 * tokens            i32[B] output (required).
 * logprobs          f32[B] output or NULL: ln p(token) under softmax(z'/T_eff) over all
 *                   allowed tokens (T_eff = 1 for rows with T < 1e-5).
 * row_status        i32[B] output or NULL.
 * dbg_transformed   f32[B, V] output or NULL: the transformed logits z' (after penalties,
 *                   bias and mask), row-major with row stride V.
 * dbg_kept_count    i32[B] output or NULL: size of the kept set K (1 for greedy rows).
 * dbg_cut           f32[B] output or NULL: min over K of y = (z' - max z') * (1/T).
 * logprobs_orig     f32[B] output or NULL: ln p(token) under softmax(z') at T = 1, the
 *                   distribution before temperature (SGLang page, "Numerical consistency
 *                   of logprobs": the original logprobs).  Costs one more exponential
 *                   per logit when requested.
 * logprobs_kept     f32[B] output or NULL: ln of the token's probability renormalised
 *                   over the kept set K, the distribution it was drawn from (GLM page,
 *                   "Sampling": the top-k/top-p sampler's processed logprobs); 0 for
 *                   greedy rows (K is the token alone).
 * tid_offs/ids      CSR of requested token ids (SGLang page, the output container's
 *                   token-ids logprobs): ids tid_ids[tid_offs[r] .. tid_offs[r+1]), in
 *                   any order, repeats allowed.  NULL offs = none.  An id outside [0, V)
 *                   or a decreasing offset makes the row INVALID.
 * tid_logprobs      f32[tid_offs[B]] output (required with tid_offs): ln p(id) under the
 *                   same distribution as `logprobs` (softmax(z'/T_eff), pre-truncation);
 *                   -inf for a masked id and for every id of an INVALID row.
 * top_ns            i32[B] or NULL: N, the number of most probable tokens to report for
 *                   row r (SGLang page, the output container's top logprobs); 0 <= N <=
 *                   min(32, top_n_stride), else the row is INVALID.  Order: probability
 *                   descending; y is monotone in z', so equal probabilities are ranked
 *                   by z' descending, then by id ascending.
 * top_n_stride      row stride (elements) of top_ids / top_logprobs, >= 1 with top_ns.
 * top_ids           i32[B, top_n_stride] output (required with top_ns): places 0..N-1 of
 *                   row r; -1 past the row's allowed tokens and for an INVALID row; places
 *                   N.. untouched.
 * top_logprobs      f32[B, top_n_stride] output (required with top_ns): ln p of those
 *                   tokens under softmax(z'/T_eff) (pre-truncation); -inf where the id is -1.
 *
 * Limits: V <= 262144 (at most 18 slices of at most 15360 tokens per row).  Any number
 * of penalised, biased or allowed tokens is handled exactly.  A row whose candidate set
 * must spill (a slice with more than 2048 candidates: flat or heavily tied rows) takes a
 * spill row for the call.  A handle has one spill row per batch row, so no valid row of
 * clsample_apply runs out; clsample_apply_static has 4, and a fifth row that must spill
 * in one of its calls gets status OVERFLOW.  A row whose bounded waits for other CTAs
 * gave up (a GPU that stopped scheduling them) is OVERFLOW too.
 */
typedef struct {
  int32_t B, V;
  int32_t logits_dtype;
  int32_t mode;
  const void* logits;
  int64_t logits_row_stride;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
  const float* rep;
  const float* freq;
  const float* pres;
  const int32_t* hist_offs;
  const int32_t* hist_ids;
  const int32_t* bias_offs;
  const int32_t* bias_ids;
  const float* bias_vals;
  const int32_t* bitmask;
  int64_t bitmask_row_stride;
  const uint64_t* seeds;
  const int64_t* positions;
  int64_t step;
  int32_t* tokens;
  float* logprobs;
  int32_t* row_status;
  float* dbg_transformed;
  int32_t* dbg_kept_count;
  float* dbg_cut;
  float* logprobs_orig;
  float* logprobs_kept;
  const int32_t* tid_offs;
  const int32_t* tid_ids;
  float* tid_logprobs;
  const int32_t* top_ns;
  int32_t top_n_stride;
  int32_t reserved1;
  int32_t* top_ids;
  float* top_logprobs;
} clsample_args_t;

/* Creates a handle for batches of up to max_batch rows over a vocabulary of `vocab`
 * tokens on the current CUDA device.  Sets the kernels' shared-memory attributes and
 * allocates the handle's device scratch (cudaMalloc; freed by clsample_destroy).
 * Returns CLSAMPLE_SUCCESS and *out, or a negative code (*out = NULL; nothing kept). */
int clsample_create(int32_t max_batch, int32_t vocab, clsample_t** out);

/* Releases a handle and its scratch (NULL is ignored).  cudaFree synchronises the
 * device, so no call on the handle may still be running. */
void clsample_destroy(clsample_t* handle);

/* Enqueues one sampler call on `stream`: the preparation launch (one CTA orders the
 * rows, heavy rows first, and resets the call's counters; when the call has penalties,
 * logit_bias or a bitmask, one more CTA per row lists the row's distinct penalised and
 * biased tokens by vocabulary slice and counts its allowed tokens), then the sampler
 * kernel (one CTA per (row, slice), launched with programmatic stream serialisation; its
 * CTAs wait, bounded, only for the flags the preparation launch sets); nothing when
 * B == 0.  Returns after enqueueing; results are valid once the stream reaches this
 * point. */
int clsample_apply(clsample_t* handle, const clsample_args_t* args, clsample_stream_t stream);

/* The two halves of clsample_apply, for callers that schedule or time them apart:
 * clsample_prepare enqueues the preparation launch, clsample_sample the sampler kernel,
 * which consumes what the last clsample_prepare on this handle wrote (each
 * clsample_sample needs its own clsample_prepare before it: the sampler clears the
 * preparation's flags when it ends; a sample without one waits a few seconds at most
 * and reports every row OVERFLOW, touching no row past B; a preparation that no sample consumes is harmless, the
 * next one clears its flags first).  The pair, with the same arguments on one stream,
 * equals clsample_apply.  Same validation and return codes. */
int clsample_prepare(clsample_t* handle, const clsample_args_t* args, clsample_stream_t stream);
int clsample_sample(clsample_t* handle, const clsample_args_t* args, clsample_stream_t stream);

/* One sampler call without a handle that allocates nothing.  The pages have no
 * counterpart: this is a deployment convenience of this library, and it samples
 * exactly like clsample_apply.  Its scratch is one fixed device array compiled into
 * the library (about 37 MB, zero when the library loads); no cudaMalloc or cudaFree
 * ever happens.  The first call on a device looks up the array's address on that
 * device (cudaGetSymbolAddress) and sets the kernels' shared-memory limit, once per
 * device, under a host lock.  Limits: B <= 64 (else CLSAMPLE_ERR_BATCH) and
 * V <= 262144 (else CLSAMPLE_ERR_VOCAB); nothing is enqueued on an error.  The array
 * holds 4 spill rows (see the limits of clsample_args_t): at most 4 rows of a call may
 * spill; a further row that must spill reports OVERFLOW.
 * Races: every call on a device, from any host thread or stream, uses the same array,
 * so calls of this entry point on one device must be ordered (one stream, or streams
 * joined by events); two overlapping calls corrupt each other's row order and records.
 * Calls through handles are unaffected, and each process has its own array. */
int clsample_apply_static(const clsample_args_t* args, clsample_stream_t stream);

/* Static description of a return code. */
const char* clsample_strerror(int code);

/* Launch geometry chosen for a vocabulary size: slices per row, tokens per slice and
 * dynamic shared memory per CTA.  Host-only; needs no GPU.  Returns CLSAMPLE_SUCCESS or
 * CLSAMPLE_ERR_VOCAB. */
int clsample_geometry(int32_t vocab, int32_t* slices, int32_t* chunk, int32_t* smem_bytes);

/* How many sampler-kernel CTAs of this handle can be resident on the device at once
 * (cudaOccupancyMaxActiveBlocksPerMultiprocessor times the SM count), computed at
 * clsample_create; the kernel launches one CTA per (row, slice). */
int clsample_occupancy(clsample_t* handle, int32_t logits_dtype, int32_t* resident_ctas);

/* Builds grammar-bitmask rows from allowed-token lists (vLLM page, "allowed token ids",
 * a hard-coded constraint of the sampler, expressed here as the bitmask the sampler
 * takes).  offs i32[B+1] and ids (DEVICE) give row r's allowed ids ids[offs[r] ..
 * offs[r+1]); bitmask i32[B, bitmask_row_stride] (DEVICE, written; words past
 * ceil(V/32) untouched) gets bit id & 31 of word id >> 5 set for each listed id and every
 * other bit cleared.  A row with an id outside [0, V), a decreasing offset or an empty
 * list ends all-zero, which clsample_apply reports as INVALID.  Enqueue only on `stream`;
 * returns a negative code for bad sizes or NULL pointers (nothing launched). */
int clsample_allowed_to_bitmask(const int32_t* offs, const int32_t* ids, int32_t B, int32_t V, int32_t* bitmask,
                                int64_t bitmask_row_stride, clsample_stream_t stream);

/* Diagnostics of the building blocks, on device arrays of length n (enqueued on
 * `stream`): the fixed-point top-p weight floor(exp32(y) * 2^40) of each y (y <= 0),
 * and the race uniform U of (seed, position, token).  They run the same device code
 * as clsample_apply, so tests can compare them with an independent implementation. */
int clsample_debug_weights(const float* y, uint64_t* weights, int32_t n, clsample_stream_t stream);
int clsample_debug_uniforms(const uint64_t* seeds, const int64_t* positions, const int64_t* tokens,
                            float* u, int32_t n, clsample_stream_t stream);

/* ------------------------------------------------------------------------------------
 * The other operators of a speculative-decoding step.  A step takes the n_b newest
 * tokens of each of B sequences (one token, the last accepted token and the drafted
 * ones, or a chunk of a prompt): clsample_kv_append writes their keys and values to a
 * paged cache, clsample_chunk_attention attends to it, the model's LM head gives the
 * verify rows, and clsample_verify accepts drafted tokens against the target's
 * probabilities.  No public page is followed here; the formulas stand with each call.
 *
 * The batch.  T token rows; sequence b owns rows cu_new[b] .. cu_new[b + 1] (int32[B + 1],
 * non-decreasing, within [0, T]; n_b may be 0; rows that no sequence owns are not
 * touched).  kv_lens[b] (int32) is the sequence's length WITH the new tokens, so row
 * cu_new[b] + i stands at position kv_lens[b] - n_b + i.
 *
 * The cache.  Two arrays of `dtype`, for keys and values, with the same strides: element
 * d of head h in slot s of page p is at p * page_stride + s * slot_stride +
 * h * head_stride + d (strides in elements, 64-bit).  Position x of sequence b is in slot
 * x % page_size of page page_table[b * table_stride + x / page_size] (int32).
 *
 * Row statuses here are per sequence: INVALID marks offsets out of order or range, a
 * negative kv_lens[b], one past max_pages * page_size, n_b > max_new, or a page id outside
 * [0, num_pages) among the pages that the call has to touch.  Nothing is read or written
 * outside the arrays; the other sequences are not affected. */

/* Element types of queries, keys, values, their cache and outputs. */
enum { CLSAMPLE_T_BF16 = 0, CLSAMPLE_T_F16 = 1 };

/* Arguments of clsample_kv_append: for each new token, in this order,
 *   1. q and k of each head: x <- x * rsqrt(mean(x^2) + eps) * weight, if weights are given;
 *   2. q and k: the first rot_dim elements are rotated by the token's position.  Pair j is
 *      (x[j], x[j + rot_dim/2]), or (x[2j], x[2j + 1]) with `interleaved`; with c =
 *      cos_sin[pos][j], s = cos_sin[pos][rot_dim/2 + j]: (a, b) <- (a c - b s, b c + a s);
 *   3. q goes to q_out, k and v to the token's slot of the cache.
 * All in float32, rounded once when stored; v is copied bit for bit.
 *
 * q, k, v           [T, heads, D] of `dtype` with token and head strides (elements).
 * q_out             like q; may be q itself (same strides).  NULL with Hq == 0.
 * cos_sin           f32[max_pos, >= rot_dim], row stride cs_stride; NULL with rot_dim 0.
 * q_weight/k_weight D elements of `dtype`, or NULL: no norm.
 * row_status        i32[B] output or NULL.
 *
 * A token whose position is negative or not below max_pos (with rotation), or whose page
 * is not valid, is not written to the cache and its q_out row is zero; its sequence is
 * INVALID.  Two tokens of a call must not share a slot.
 * Limits: 1 <= D <= 256, rot_dim even and <= D, any strides, lengths up to 2^30.  Fast path: D, rot_dim (and
 * rot_dim/2 in the half-split form) multiples of 8, arrays and strides multiples of 16 bytes,
 * at most 256 heads in all. */
typedef struct {
  int32_t B, T, Hq, Hkv, D;
  int32_t dtype;
  int32_t num_pages, page_size, max_pages;
  int32_t rot_dim, max_pos, interleaved;
  float eps;
  int32_t reserved0;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_cache;
  void* v_cache;
  int64_t q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h, qo_stride_t, qo_stride_h;
  int64_t page_stride, slot_stride, head_stride;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* cu_new;
  const int32_t* kv_lens;
  const float* cos_sin;
  int64_t cs_stride;
  const void* q_weight;
  const void* k_weight;
  int32_t* row_status;
} clsample_kv_append_args_t;

/* Enqueues one append on `stream` (one launch; none when T == 0 or B == 0, except that
 * the statuses of B sequences without tokens are written).  No handle, no scratch; the arrays
 * are the current device's. */
int clsample_kv_append(const clsample_kv_append_args_t* args, clsample_stream_t stream);

/* Arguments of clsample_chunk_attention.  Query head h reads key head h / (Hq / Hkv).  The
 * row at position x sees the keys at positions <= x, of those only the last `window` when
 * window > 0:
 *   out = sum_j softmax_j(scale * q . k_j) v_j,   lse = ln sum_j exp(scale * q . k_j).
 * A row that sees no key (kv_lens[b] < n_b) gets out 0 and lse -inf.  Slots that no row of
 * the sequence sees may hold anything: those of a page with others that are seen may be read, but
 * nothing depends on them.  Ids of pages without a slot that is seen are not looked at.
 *
 * q, out            [T, Hq, D] of `dtype`, token and head strides (elements).
 * lse               f32[T, Hq] output or NULL.
 * max_new           upper bound of n_b, known to the caller; a sequence above it is
 *                   INVALID and its out rows are 0.  It also chooses the kernels: only up to
 *                   16 packed rows (max_new Hq / Hkv) does a call take the one for few rows
 *                   alone, so a loose bound costs decoding batches time, and results of
 *                   different bounds may differ in their rounding.
 * scale             in (0, 2e38] (1 / sqrt(D) as a rule).
 * row_status        i32[B] output or NULL.  Keys on a page with an invalid id are left out.
 *
 * Products are of `dtype` with float32 sums; the softmax is float32; its weights are
 * rounded to `dtype` for the product with the values, as the matrix instructions need.
 * The result of a call does not depend on timing: partial sums over a split key axis are
 * joined in key order.  A value that is not finite, of a key that a row does not see but another
 * new row of the sequence does, may make the first row NaN (0 x NaN in a product).
 * A wait inside the kernels that runs out (about two seconds; a GPU that stopped scheduling them)
 * does not hang: the call ends, all sequences of that call and of later calls on the handle are
 * OVERFLOW, and what that call wrote to its rows of out and lse is void.
 * Limits: D 64 or 128; Hq a multiple of Hkv; q, out and cache addresses and strides
 * multiples of 16 bytes (ERR_ALIGN); T Hq / Hkv below 2^31 - 1024; lengths up to 2^30.
 * Speed: pages of 8, 16, 32, 64 or a multiple of 128 slots are copied by TMA for sequences of
 * more than 16 packed rows (n_b Hq / Hkv); other sizes take about twice the time there. */
typedef struct {
  int32_t B, T, Hq, Hkv, D;
  int32_t dtype;
  int32_t num_pages, page_size, max_pages;
  int32_t max_new, window;
  float scale;
  const void* q;
  void* out;
  const void* k_cache;
  const void* v_cache;
  int64_t q_stride_t, q_stride_h, o_stride_t, o_stride_h;
  int64_t page_stride, slot_stride, head_stride;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* cu_new;
  const int32_t* kv_lens;
  float* lse;
  int32_t* row_status;
} clsample_attention_args_t;

/* A handle holds the device scratch in which partial sums of a split key axis meet: its
 * size depends on the device alone, not on any call.  Bound to the device that was current;
 * calls on one handle must be ordered, as for clsample_t. */
typedef struct clsample_attention clsample_attention_t;
int clsample_attention_create(clsample_attention_t** out);
void clsample_attention_destroy(clsample_attention_t* handle);

/* Enqueues one call on `stream` (two or three launches, each of which may start while the one
 * before it ends; they can be captured in a graph); nothing when B == 0. */
int clsample_chunk_attention(clsample_attention_t* handle, const clsample_attention_args_t* args,
                             clsample_stream_t stream);

/* Test hook.  In later calls on the handle a barrier of the kernel for more than 16 packed rows
 * waits for one arrival more than it gets, and no wait takes more than wait_cycles (1 to 4e9) SM
 * cycles.  barrier: the unit of work (1) and its end (2), its queries (3) and their end (4), keys
 * copied (5) and handed over (6), values copied (7) and handed over (8), a tile's end (9), its scores
 * (10), half of its weights (11), all of them (12), the sums (13); slot: which of several.  0: none,
 * which is also how a handle starts. */
int clsample_debug_attention_stall(clsample_attention_t* handle, int32_t barrier, int32_t slot, int64_t wait_cycles);

/* Arguments of clsample_verify.  Request b drafted n_b = cu_draft[b + 1] - cu_draft[b] >= 0
 * tokens (cu_draft int32[B + 1], within [0, N]).  Its n_b + 1 rows of target probabilities
 * start at row cu_draft[b] + b of `target` (N + B rows); its draft probabilities are rows
 * cu_draft[b] .. of `draft` (N rows; NULL when the draft is certain of its tokens, q = 1).
 *   1. Drafted tokens x_i are accepted in order while u_i q_i(x_i) < p_i(x_i), u_i =
 *      u_accept[cu_draft[b] + i] (the two sides are compared exactly).
 *   2. One more token is drawn with u = u_sample[b]: at the first refusal from the weights
 *      max(P_i(t) - Q_i(t), 0), P = floor(p 2^40) and Q = floor(q 2^40) (Q = 2^40 at x_i
 *      for a certain draft, 0 elsewhere); if none was refused, or if all those weights are
 *      0, from P.  With W their sum, the token is the lowest t whose inclusive running
 *      sum is above floor(floor(u 2^31) W / 2^31).  All in integers: the result does not
 *      depend on how the row is split.
 * The tokens kept are distributed as the target's own (the standard argument: min(p, q) +
 * max(p - q, 0) = p).  A greedy target is a row with 1 at its token.
 *
 * target, draft     [rows, V] probabilities of `dtype` (CLSAMPLE_LOGITS_F32 or _BF16), row
 *                   strides >= V (elements).  They need not sum to 1.
 * draft_tokens      i32[N].   u_accept f32[N], u_sample f32[B], in [0, 1).
 * tokens            i32[B, token_stride] output, token_stride > max_draft: accepted tokens,
 *                   the drawn token, then -1 up to place max_draft.
 * accepted          i32[B] output or NULL: how many drafted tokens were accepted.
 * row_status        i32[B] output or NULL.  INVALID (tokens all -1, accepted 0): offsets out
 *                   of order or range, n_b > max_draft, a token outside [0, V), a random
 *                   number outside [0, 1), a probability outside [0, 1] or NaN where the
 *                   call reads one (at the drafted tokens, and in the rows it draws from),
 *                   or a row to draw from without mass.
 * Limits: 0 < V <= 262144. */
typedef struct {
  int32_t B, N, V;
  int32_t dtype;
  int32_t max_draft, reserved0;
  const void* target;
  int64_t target_stride;
  const void* draft;
  int64_t draft_stride;
  const int32_t* draft_tokens;
  const int32_t* cu_draft;
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens;
  int64_t token_stride;
  int32_t* accepted;
  int32_t* row_status;
} clsample_verify_args_t;

/* Enqueues one verification on `stream` (one launch); nothing when B == 0.  No handle, no scratch;
 * the arrays are the current device's. */
int clsample_verify(const clsample_verify_args_t* args, clsample_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* CLSAMPLE_H */
