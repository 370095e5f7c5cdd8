/*
 * svw.h -- C ABI of the vocabulary-wide speculative-verification library
 * (serving_vocab_wide_gb300).  Hand-written CUDA for sm_103a (GB300).
 *
 * Two operations, both over full-vocabulary logits (and spec_verify_opd,
 * both on the same batch in one pass), two variants of the verification
 * (spec_verify_early: stops reading each request at its first rejection;
 * spec_verify_filtered: top-k / top-p filtered distributions), plus the
 * adaptive length head that sets the next round's verified lengths
 * (length_head, length_head_label), and the steps of a round that precede the
 * verification (kv_append, paged_attention, logits_adjust; kv_append_norm,
 * paged_attention_fp8 and kv_gather with a cache of 8 bits):
 *
 *  spec_verify  batched speculative verification of a ragged batch.  Defined
 *               by "DFlash 阅读笔记：并行起草、目标特征与精确验证" §5.1 (greedy
 *               rule), §5.2 eqs. (6)-(8) and Algorithm 1, and by "AdaFlash:
 *               Taming Variance in Diffusion Speculative Decoding", section
 *               "Speculative Decoding: The Basic Idea", steps 3-4.  Requests
 *               are packed by CSR offsets ("AdaFlash：基于在策略蒸馏扩散草稿器
 *               的自适应投机解码" §2.3: the verify batch holds each request's
 *               own length, not N x k).
 *
 *  opd_loss     entry-wise clipped reverse KL(q||p) + lambda * CE on the
 *               target top-1 token, and its gradient wrt the draft logits.
 *               Defined by "AdaFlash: Taming Variance in Diffusion Speculative
 *               Decoding", sections "The Reverse-KL + Hard-Label Mixture Loss,
 *               Derived" and "Algorithm 2: Entry-Wise Clipped Reverse-KL".
 *
 * Conventions for every entry point:
 *  - Pointers named "device" are CUDA device pointers (cudaMalloc / PyTorch
 *    CUDA tensors) on the current device.  The caller owns all memory; the
 *    library allocates and frees no device memory and keeps no per-call state
 *    (length_head's GEMM library keeps a host handle and per-shape plans).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Calls are stream-ordered and never synchronise the host.
 *  - The return value covers host-side validation and launch errors only.
 *    Problems that only the device can see (bad CSR offsets, out-of-range
 *    tokens, non-finite rows) are reported by OR-ing SVW_DEV_* bits into
 *    *status (device int32, may be NULL); the caller clears it.
 *  - Logits are row-major [rows, V] in fp32 or bf16.  Rows whose byte pitch
 *    V * sizeof(dtype) is a multiple of 16 with 16-byte aligned bases take the
 *    vectorised / bulk-copy path; any other shape takes a scalar path with the
 *    same results.
 *  - Inputs are read-only; outputs must not alias inputs, except where an
 *    entry point says so (logits_adjust, kv_append's and kv_append_norm's queries).
 */
#ifndef SVW_H_
#define SVW_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum svw_status {
  SVW_OK = 0,
  SVW_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, bad temperature ... */
  SVW_ERR_UNSUPPORTED = 2, /* dtype or size outside what the kernels handle         */
  SVW_ERR_UNSUPPORTED_DTYPE = SVW_ERR_UNSUPPORTED, /* the same code, by its other name */
  SVW_ERR_MISALIGNED = 3,  /* a pointer violates its documented alignment            */
  SVW_ERR_WORKSPACE = 4,   /* workspace missing or smaller than its *_workspace_size  */
  SVW_ERR_CUDA = 5,        /* a CUDA runtime call or kernel launch failed            */
  SVW_ERR_BAD_INPUT = 6,   /* device-detected: see svw_device_status()               */
  SVW_ERR_TIMEOUT = 7      /* device-detected: see svw_device_status()               */
} svw_status;

/* SVW_E4M3: 8-bit floats (4 bits of exponent, 3 of mantissa, largest 448, no
 * infinity), the type of a cache where an entry point says so. */
typedef enum svw_dtype { SVW_F32 = 0, SVW_BF16 = 1, SVW_E4M3 = 2 } svw_dtype;

/*
 * Bits OR-ed into the device status word.  The word is a bit set, not an
 * svw_status: many CTAs of one call may each find a problem, and an atomic OR
 * of bits is the only way they can report without ordering.  No entry point
 * returns SVW_ERR_BAD_INPUT or SVW_ERR_TIMEOUT from the host (the host never
 * waits for the device); svw_device_status() turns a word the caller has read
 * back into those codes.
 */
#define SVW_DEV_BAD_INPUT 1 /* some request / row was invalid or non-finite   */
#define SVW_DEV_TIMEOUT 2   /* a bounded wait inside a kernel gave up         */

/*
 * The svw_status of a device status word read back by the caller:
 * SVW_ERR_TIMEOUT if SVW_DEV_TIMEOUT is set (results of that call are not
 * valid), else SVW_ERR_BAD_INPUT if SVW_DEV_BAD_INPUT is set (the bad
 * requests / rows carry -1 / NaN, the others are valid), else SVW_OK.
 */
svw_status svw_device_status(int32_t status_word);

/* Largest draft length (positions per request) spec_verify accepts. */
#define SVW_MAX_LEN 32

/*
 * svw_workspace_size -- one workspace size for every entry point that verifies
 * or distils a batch shape (the steps before a verification, logits_adjust and
 * paged_attention, have their own): the largest of svw_verify_workspace_size, svw_verify_early_workspace_size,
 * svw_verify_filtered_workspace_size (both dtypes), svw_opd_workspace_size and
 * svw_verify_opd_workspace_size for (n_requests, total_draft_rows, V), so
 * that a caller can size one buffer before it knows which call or dtype it
 * will make.  max_len (1..SVW_MAX_LEN) is checked only.  Returns 0 for
 * invalid arguments.  The per-call functions below give the exact (smaller)
 * sizes.
 */
size_t svw_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V, int32_t max_len);

/*
 * Bytes of device workspace spec_verify needs for this batch shape (any
 * temperature).  Depends only on (n_requests, total_draft_rows, V, dtype).
 * Returns 0 for invalid arguments.
 */
size_t svw_verify_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V,
                                 svw_dtype dtype);

/*
 * spec_verify -- verify every request of a ragged batch in one call.
 *
 * Request i owns L_i = cu_draft[i+1] - cu_draft[i] draft positions.
 *   draft_logits  device [total_draft_rows, V]; request i's rows are
 *                 cu_draft[i] .. cu_draft[i+1]-1 (position j at cu_draft[i]+j).
 *   target_logits device [total_draft_rows + N, V]; request i's rows are
 *                 cu_draft[i]+i .. cu_draft[i]+i+L_i: row j is the target's
 *                 distribution at draft position j, the last (j = L_i) is the
 *                 bonus row used when every candidate passes.
 *   cu_draft      device int32 [N+1], cu_draft[0] = 0, non-decreasing,
 *                 cu_draft[N] = total_draft_rows (passed on the host so that
 *                 the call never reads device memory from the host).
 *   max_len       1..SVW_MAX_LEN; requests with L_i outside [1, max_len] are bad.
 *   draft_tokens  device int32 [total_draft_rows], x_j drawn from
 *                 softmax(draft row j / temperature); must be in [0, V).
 *   temperature   0 => greedy: accept x_j iff it is the target argmax of row j
 *                 (raw logits, smallest index wins); next_token is the argmax
 *                 of the first rejected row, or of the bonus row.
 *                 > 0 => accept x_j iff u_j < min(1, p_j(x_j) / q_j(x_j)) with
 *                 p = softmax(target/T), q = softmax(draft/T); the accepted
 *                 length is the leftmost-rejection prefix; next_token is drawn
 *                 by inverse CDF (vocabulary order, smallest v with C_v > w Z)
 *                 from max(0, p - q) at the rejected row, or from p at the
 *                 bonus row.
 *   seed          Philox4x32-10 key (lo 32 bits, hi 32 bits).  u_j uses counter
 *                 {i, j, 0, 0}; the sampling uniform w uses {i, j*, 1, 0}, j*
 *                 the sampled row.  Uniform = (word0 >> 8) * 2^-24.
 *   accept_len    device int32 [N] out; -1 for a bad request.
 *   next_token    device int32 [N] out; -1 for a bad request.
 *   status        device int32 scalar, may be NULL; SVW_DEV_BAD_INPUT is
 *                 OR-ed in if any request is bad (invalid length, token out of
 *                 range, a NaN row, or at T > 0 a row with +Inf or only -Inf).
 *   workspace     device, 256-byte aligned, >= svw_verify_workspace_size(...)
 *                 bytes; contents need not be initialised; not preserved.
 */
svw_status spec_verify(const void *target_logits, const void *draft_logits, svw_dtype dtype,
                       int32_t V, int32_t N, const int32_t *cu_draft, int64_t total_draft_rows,
                       int32_t max_len, const int32_t *draft_tokens, float temperature,
                       uint64_t seed, int32_t *accept_len, int32_t *next_token, int32_t *status,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * spec_verify_early -- spec_verify that stops reading a request at its first
 * rejection.
 *
 * Leftmost rejection ("DFlash 阅读笔记：并行起草、目标特征与精确验证" §5.2,
 * Algorithm 1) makes every row after a request's first rejected position
 * irrelevant to its result, and acceptance falls with the position
 * ("AdaFlash：基于在策略蒸馏扩散草稿器的自适应投机解码" §3.3, Figure 2(c):
 * from about 0.9 at the first position to 0.13-0.26 at the fifteenth).  The
 * rows are streamed position by position across the batch and each accept
 * test runs as soon as its two rows are reduced; rows at positions after a
 * known rejection are skipped.  Which later rows still get read depends on
 * timing, the results do not.
 *
 * Arguments and results as for spec_verify (same accept_len and next_token,
 * bit for bit, same uniforms), with these differences:
 *   - a request is bad (accept_len = next_token = -1) if a row at or before
 *     its first rejected position (the bonus row when none is rejected) is
 *     non-finite, or if any of its tokens is out of range; rows after the
 *     first rejection are not checked (they need not be read);
 *   bytes_read    device uint64 scalar out, may be NULL: the logit bytes this
 *                 call streamed from the two tensors (without the one row
 *                 pair the draw reads again).  Reset by the call.  8-byte
 *                 aligned.
 *   workspace     >= svw_verify_early_workspace_size(...) bytes.
 */
size_t svw_verify_early_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V,
                                       svw_dtype dtype);

svw_status spec_verify_early(const void *target_logits, const void *draft_logits, svw_dtype dtype, int32_t V,
                             int32_t N, const int32_t *cu_draft, int64_t total_draft_rows, int32_t max_len,
                             const int32_t *draft_tokens, float temperature, uint64_t seed, int32_t *accept_len,
                             int32_t *next_token, int32_t *status, unsigned long long *bytes_read,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Largest top_k spec_verify_filtered accepts. */
#define SVW_FILTER_MAX_K 1024

/*
 * spec_verify_filtered -- spec_verify with both distributions top-k / top-p
 * filtered.
 *
 * The pages verify with the full temperature softmax; serving stacks usually
 * filter first.  This variant is not on the pages and follows this reading:
 * p and q are filtered with the same (temperature, top_k, top_p) -- entries
 * ordered by raw logit descending, the smaller index first among equal
 * logits; the first top_k kept; of those, the shortest prefix whose
 * probability reaches top_p times their total kept; renormalised -- and the
 * method of spec_verify ("DFlash 阅读笔记：并行起草、目标特征与精确验证" §5.2
 * eqs. (6)-(8), Algorithm 1) runs on the filtered p' and q': x_j is accepted
 * iff u_j < min(1, p'(x_j) / q'(x_j)) (a token outside the target's kept set
 * is rejected; q'(x_j) = 0 with p'(x_j) > 0 is accepted), the next token is
 * drawn from [p' - q']_+ at the rejected row or from p' at the bonus row, by
 * the same inverse CDF in vocabulary order.  draft_tokens are drawn from q'.
 *
 * Arguments and results as for spec_verify, plus:
 *   top_k         1 .. SVW_FILTER_MAX_K (a larger value returns
 *                 SVW_ERR_UNSUPPORTED; values >= V keep every entry).
 *   top_p         (0, 1]; 1 keeps the whole top-k set.
 *   temperature   0 => greedy spec_verify (filtering keeps the argmax).
 *   workspace     >= svw_verify_filtered_workspace_size(...) bytes.
 * V is limited by shared memory (about 200 KB per CTA: V <= ~600 k for bf16
 * at top_k <= 256); larger rows return SVW_ERR_UNSUPPORTED.
 */
size_t svw_verify_filtered_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V,
                                          svw_dtype dtype);

svw_status spec_verify_filtered(const void *target_logits, const void *draft_logits, svw_dtype dtype, int32_t V,
                                int32_t N, const int32_t *cu_draft, int64_t total_draft_rows, int32_t max_len,
                                const int32_t *draft_tokens, float temperature, int32_t top_k, float top_p,
                                uint64_t seed, int32_t *accept_len, int32_t *next_token, int32_t *status,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * opd_loss -- per draft row r (0 <= r < total_draft_rows), paired with one
 * target row:
 *   lp = log softmax(target/T), lq = log softmax(draft/T), q = exp(lq)
 *   t_v = q_v (lq_v - lp_v)          (t_v := 0 where q_v = 0)
 *   loss[r] = sum_v clamp(t_v, -clip_c, clip_c) + lambda_ce * (-lq[x*]),
 *             x* = argmax of the raw target row (smallest index wins)
 *   dlogits[r, v] = grad_scale / T * ( q_v (a_v - S) + lambda_ce (q_v - [v == x*]) ),
 *             a_v = [-clip_c < t_v < clip_c] (lq_v - lp_v + 1), S = sum_v q_v a_v
 * i.e. dlogits is grad_scale times the gradient of sum_r loss[r] wrt the
 * draft logits (the target is frozen).  Pass grad_scale = 1/k for the mean
 * over k positions.
 *
 *   target_has_bonus_row  1: verify layout -- target has total_draft_rows + N
 *                 rows and draft row r of request i pairs with target row r + i
 *                 (cu_draft device [N+1] required).  0: rows pair 1:1, target
 *                 has total_draft_rows rows, cu_draft and N are ignored.
 *   temperature   > 0 (the reverse-KL temperature; 1.0 in the review).
 *   clip_c        > 0 (may be +inf: no clipping).
 *   loss          device float [total_draft_rows] out (NaN for a bad row).
 *   dlogits       device float [total_draft_rows, V] out, 16-byte aligned;
 *                 NULL computes the loss only.
 *   status        as for spec_verify (SVW_DEV_BAD_INPUT for a non-finite row
 *                 or a row outside its request's CSR range; SVW_DEV_TIMEOUT if
 *                 a bounded wait on a bulk copy gave up).
 *   workspace     device, 256-byte aligned, >= svw_opd_workspace_size(
 *                 total_draft_rows) bytes (per row: a flag, the row
 *                 constants, 128 partial clamped sums; about 1 KB), contents
 *                 need not be initialised, not preserved; or NULL.  With a
 *                 workspace, rows whose byte pitch is a multiple of 16 take
 *                 a one-exchange fast pass, which also leaves each row's
 *                 exact clamped sum as partials, and only the gradient of
 *                 rows where some term reaches the clip (or the draft has
 *                 masked entries) is written again; the results are the same
 *                 either way (up to float rounding order).
 */
size_t svw_opd_workspace_size(int64_t total_draft_rows);

svw_status opd_loss(const void *target_logits, const void *draft_logits, svw_dtype dtype,
                    int32_t V, int32_t N, const int32_t *cu_draft, int64_t total_draft_rows,
                    int32_t target_has_bonus_row, float temperature, float clip_c,
                    float lambda_ce, float grad_scale, float *loss, float *dlogits,
                    int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/*
 * spec_verify_opd -- spec_verify and opd_loss (verify layout) on the same
 * batch in one pass over the logits.  The distillation signal is a byproduct
 * of verification ("AdaFlash: Taming Variance in Diffusion Speculative
 * Decoding", "Method Part 1: On-Policy Distillation (OPD) for Diffusion
 * Drafters", "Algorithm, Step by Step" step 3 and Figure 2: the target's
 * distribution at every drafted position is already computed by
 * verification), so both results come from one read of both logit tensors:
 * the OPD kernel's row softmaxes serve the accept tests, and the bonus rows
 * are reduced in the same pass.
 *
 * Arguments as for spec_verify and opd_loss, plus:
 *   temperature      verification temperature (0: greedy).
 *   opd_temperature  > 0, the reverse-KL temperature; must equal temperature
 *                    when temperature > 0 (the softmaxes are shared), else
 *                    SVW_ERR_INVALID_ARG.
 *   loss, dlogits    as for opd_loss with target_has_bonus_row = 1.
 *   workspace        device, 256-byte aligned, >= svw_verify_opd_workspace_size
 *                    bytes; contents need not be initialised; not preserved.
 * accept_len / next_token equal spec_verify's and loss / dlogits equal
 * opd_loss's on the same inputs, with one difference: a request with a
 * non-finite row (NaN, +Inf, or only -Inf in any of its target, bonus or
 * draft rows) is reported bad at every temperature (spec_verify at T = 0
 * only rejects NaN target rows).  Needs 16-byte aligned bases and a 16-byte
 * row pitch (V * sizeof(dtype) % 16 == 0) and a row the one-pass kernel can
 * hold on chip (V = 151936 bf16 fits); otherwise SVW_ERR_UNSUPPORTED.
 */
size_t svw_verify_opd_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V,
                                     svw_dtype dtype);

svw_status spec_verify_opd(const void *target_logits, const void *draft_logits, svw_dtype dtype,
                           int32_t V, int32_t N, const int32_t *cu_draft, int64_t total_draft_rows,
                           int32_t max_len, const int32_t *draft_tokens, float temperature,
                           float opd_temperature, uint64_t seed, float clip_c, float lambda_ce,
                           float grad_scale, int32_t *accept_len, int32_t *next_token, float *loss,
                           float *dlogits, int32_t *status, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * length_head -- the adaptive length head's forward pass ("AdaFlash: Taming
 * Variance in Diffusion Speculative Decoding", "Algorithm 3: Adaptive Length
 * Head, Forward Pass"; "AdaFlash：基于在策略蒸馏扩散草稿器的自适应投机解码" §2.2):
 * for each request i, from its drafter hidden states h_i (k positions x H),
 *   h'_p = SiLU(W1 h_i[p] + b1),  hbar = (1/k) sum_p h'_p,
 *   a_hat[i] = sigmoid(w2 . hbar + b2),
 *   k_hat[i] = clamp(floor(gamma a_hat[i] k), 1, k)   (next round's verified length).
 *   hidden     device bf16 [N, k, H] row-major, 16-byte aligned, H % 8 == 0;
 *              N k <= 2^20 positions and k <= SVW_MAX_LEN (else
 *              SVW_ERR_UNSUPPORTED, and a workspace size of 0).
 *   w1         device bf16 [hidden_out, H] row-major (H' = hidden_out < H).
 *   b1, w2     device float [hidden_out];  b2, gamma > 0 on the host.
 *   a_hat      device float [N] out (before the gamma scaling);  k_hat device int32 [N] out.
 *   workspace  device, 256-byte aligned, >= svw_length_head_workspace_size(N, k,
 *              hidden_out) bytes: one fp32 per position and 256-wide column
 *              tile of W1 (N k ceil(H'/256) floats, rounded up to 256 bytes);
 *              contents need not be initialised.
 * The projection of the N k positions runs on the tensor cores (tcgen05 MMA,
 * operands staged by TMA, fp32 accumulation in tensor memory) in four K
 * quarters, one thread-block cluster per 128 positions; the quarters are
 * summed inside the cluster (distributed shared memory), and the same kernel
 * applies bias and SiLU and dots each position with w2.  A second, small
 * kernel adds each request's position dots and applies the mean, b2,
 * sigmoid, gamma, floor and clamp.  Two kernel launches, each a programmatic
 * dependent of the one ahead (its set-up overlaps that kernel's tail); no
 * library call; the host only encodes the two TMA descriptors.  If a bounded
 * wait inside the projection gives up, the affected requests get a_hat = NaN.
 */
size_t svw_length_head_workspace_size(int32_t n_requests, int32_t k, int32_t hidden_out);

svw_status length_head(const void *hidden, const void *w1, const float *b1, const float *w2, float b2,
                       int32_t N, int32_t k, int32_t H, int32_t hidden_out, float gamma, float *a_hat,
                       int32_t *k_hat, void *workspace, size_t workspace_bytes, void *stream);

/*
 * length_head_label -- the length head's training signal ("AdaFlash: Taming
 * Variance in Diffusion Speculative Decoding", "Online Update of the Length
 * Head, Derived"): a_star[i] = accept_len[i] / L_i, the accepted fraction of
 * the L_i = cu_draft[i+1] - cu_draft[i] verified tokens, and (loss not NULL)
 * loss[i] = (a_hat[i] - a_star[i])^2.  A bad request (accept_len < 0) gets
 * NaN.  All pointers device; a_hat may be NULL when loss is NULL.
 */
svw_status length_head_label(const int32_t *accept_len, const int32_t *cu_draft, const float *a_hat, int32_t N,
                             float *a_star, float *loss, void *stream);

/*
 * The steps around a verification on the same ragged batch: the target's
 * forward pass writes the new tokens' keys and values into a paged cache
 * (kv_append), attends from them (paged_attention), and its logits are
 * adjusted (logits_adjust) before spec_verify reads them ("AdaFlash：基于在策略
 * 蒸馏扩散草稿器的自适应投机解码" §2.3: the verified positions of all requests
 * are packed, sum of L_i + 1 tokens, without padding).  No counterpart on the
 * pages; the formulas below are the definitions.
 */

/*
 * logits_adjust -- penalties for repeated tokens, biases and grammar masks on
 * the logits of every drafted position.
 *
 * Row j of request i (0 <= j < L_i, and j = L_i when has_bonus_row) has seen
 * the request's history and its drafted tokens x_0 .. x_{j-1}.  With
 * n(v) = the occurrences of v in the history after its first prompt_len[i]
 * tokens and in that drafted prefix, and seen(v) = n(v) > 0 or v in the
 * prompt part, in fp32 and in this order:
 *   y = logits[row, v]
 *   seen(v):  y = y > 0 ? y / repetition[i] : y * repetition[i]
 *   n(v) > 0: y = y - frequency[i] n(v) - presence[i]
 *   v listed in the request's biases: y = y + its value (the last one listed)
 *   mask bit of v is 0: y = -inf (whatever y is, NaN too)
 * rounded once to the logits' type; an entry that none of these touches is
 * copied bit for bit.  A row whose mask allows nothing is all -inf (which
 * spec_verify reports as a bad request at T > 0).
 *
 *   logits         device [rows, V], row pitch logits_stride elements (>= V);
 *                  rows = total_draft_rows (+ N when has_bonus_row), request
 *                  i's first row at cu_draft[i] (+ i).
 *   cu_draft       device int32 [N+1], as for spec_verify; 0 <= L_i <=
 *                  SVW_MAX_LEN (L_i = 0 with has_bonus_row: a request that
 *                  decodes one token without a draft).
 *   draft_tokens   device int32 [total_draft_rows]; may be NULL when that is 0.
 *   history        device int32 [total_history], request i's tokens at
 *                  cu_history[i] .. cu_history[i+1]-1; cu_history NULL: none.
 *   prompt_len     device int32 [N], 0 <= prompt_len[i] <= its history's
 *                  length; NULL: 0.
 *   repetition     device float [N], finite and > 0; NULL: 1.
 *   frequency, presence  device float [N], finite; NULL: 0.
 *   bias_tokens, bias_values  device int32 / float [total_bias], request i's
 *                  at cu_bias[i] .. cu_bias[i+1]-1; values < +inf (-inf bans
 *                  the token); cu_bias NULL: none.
 *   mask           device uint32 [mask_rows, ceil(V / 32)], bit v % 32 of
 *                  word v / 32 set: v is allowed; NULL: none.
 *   mask_row       device int32 [rows]: the mask row of each logit row, -1:
 *                  unmasked; NULL: row r has mask row r (mask_rows = rows).
 *   out            device [rows, V], row pitch out_stride; equal to logits
 *                  (same pitch): in place, only what changes is written.  Any
 *                  other overlap of the two ranges is SVW_ERR_INVALID_ARG.
 *   status         as for spec_verify; SVW_DEV_BAD_INPUT when a request's
 *                  lists are inconsistent, hold a token outside [0, V) or a
 *                  factor outside its range (its rows become NaN, which
 *                  spec_verify reports as a bad request), a mask row is
 *                  outside [-1, mask_rows) (that row becomes NaN), or its
 *                  CSR range is invalid (its rows are not written).
 *   workspace      device, 256-byte aligned, >= svw_logits_adjust_workspace_size
 *                  bytes (0: none is needed); contents need not be
 *                  initialised; not preserved; or NULL.  With it the lists of
 *                  a large batch are counted once per request instead of once
 *                  per 4096 entries of its vocabulary; the results are the
 *                  same.  (Where offsets run backwards, requests that begin
 *                  inside an earlier one's lists are bad too with it.)
 */
size_t svw_logits_adjust_workspace_size(int32_t n_requests, int32_t V, int64_t total_draft_rows, int64_t total_history,
                                        int64_t total_bias);

svw_status logits_adjust(const void *logits, int64_t logits_stride, svw_dtype dtype, int32_t V, int32_t N,
                         const int32_t *cu_draft, int64_t total_draft_rows, int32_t has_bonus_row,
                         const int32_t *draft_tokens, const int32_t *history, const int32_t *cu_history,
                         int64_t total_history, const int32_t *prompt_len, const float *repetition,
                         const float *frequency, const float *presence, const int32_t *bias_tokens,
                         const float *bias_values, const int32_t *cu_bias, int64_t total_bias,
                         const uint32_t *mask, int64_t mask_rows, const int32_t *mask_row, void *out,
                         int64_t out_stride, int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/*
 * A paged key / value cache: n_pages pages of page_size tokens for each of
 * n_kv_heads heads of head_dim elements.  Element e of head h of the token in
 * row r of page p is at p * stride[0] + h * stride[1] + r * stride[2] + e
 * (strides in elements, so that pages may hold heads of tokens or tokens of
 * heads).  A request's tokens lie in the pages of its row of the block table:
 * token t in page block_table[i * table_stride + t / page_size], row
 * t % page_size.  Entries of pages that no token of the request needs may
 * hold anything.
 */
typedef struct svw_paged_kv {
  void *k;
  void *v;
  int64_t k_stride[3];
  int64_t v_stride[3];
  const int32_t *block_table; /* device int32 [N, max_pages], row pitch table_stride */
  int64_t table_stride;
  int32_t max_pages;
  int32_t n_pages;
  int32_t page_size;
  int32_t n_kv_heads;
  int32_t head_dim;
} svw_paged_kv;

/*
 * kv_append -- the new tokens' keys, rotated by their positions, and values
 * written to the paged cache; optionally their queries rotated too.
 *
 * Request i owns the new tokens cu_new[i] .. cu_new[i+1]-1 (n_i of them, 0
 * allowed); they are its last ones: token t sits at place
 * kv_len[i] - n_i + t of the cache, kv_len[i] counting the new tokens.  The
 * position rotated by is that place, or positions[token].  With c, s the
 * first and second half of cos_sin's row of that position, pair u of
 * 0 .. rot_dim/2 - 1 of each head of k (and q) becomes
 *   (a, b) -> (a c_u - b s_u, b c_u + a s_u)        (fp32, rounded once)
 * with (a, b) the elements (u, u + rot_dim/2), or (2u, 2u + 1) when
 * interleaved; elements from rot_dim on are copied, as is all of v.
 *
 *   k, v       device [total_new, n_kv_heads, head_dim], of type dtype as the
 *              cache is; strides of tokens and heads in elements (those of
 *              dimensions of one do not count).
 *   q, q_out   device [total_new, n_q_heads, head_dim], q strided like k,
 *              q_out contiguous; both NULL: no queries.  q_out may be q
 *              itself when q is contiguous.
 *   cu_new     device int32 [N+1], cu_new[0] = 0, cu_new[N] = total_new.
 *   cos_sin    device float [max_pos, rot_dim]; NULL with rot_dim = 0: no
 *              rotation.  rot_dim even, <= head_dim <= 1024.
 *   status     SVW_DEV_BAD_INPUT when a token is in no request's valid range
 *              of new tokens, its place is negative or beyond its block table,
 *              its page is not one of the cache's, or its position is outside
 *              [0, max_pos): such a token is not written (its query, if its
 *              position is bad, becomes NaN).
 * Two new tokens never share a place; pages shared by requests must not be
 * written.  One kernel launch, no workspace.
 */
svw_status kv_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                     int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
                     int64_t q_head_stride, void *q_out, svw_dtype dtype, int32_t n_q_heads, int32_t N,
                     const int32_t *cu_new, int64_t total_new, const int32_t *kv_len, const int32_t *positions,
                     const float *cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                     const svw_paged_kv *cache, int32_t *status, void *stream);

/*
 * kv_append_norm -- kv_append with a norm of each head of keys and queries
 * ahead of the rotation, into a cache of the new tokens' type or of 8 bits.
 *
 * In fp32, for each head x of a token's keys (queries likewise, with q_weight):
 *   y_e = x_e k_weight_e / sqrt(mean_e x_e^2 + eps)       (k_weight NULL: y = x)
 * its pairs rotated as kv_append's are.  Into a cache of SVW_E4M3 a key of head
 * h is written as the code nearest to y / k_scale[h], a value as the one nearest
 * to v / v_scale[h] (the quotients in fp32; ties to even; beyond +-448,
 * infinities too: +-448; NaN: NaN), so that code x scale stands for it; into a
 * cache of dtype as it is.  Rounded once.  Shapes and alignments that take the
 * scalar path add and multiply in another order: a normed or rotated number may
 * differ there by fp32's roundings, and so by a step of its type.
 *
 * Arguments and results as for kv_append, except:
 *   k_weight, q_weight  device float [head_dim]; NULL: no norm.  q_weight needs q.
 *   eps          finite, >= 0.
 *   cache_dtype  dtype or SVW_E4M3.  The cache's strides count its elements.
 *   k_scale, v_scale  device float [n_kv_heads], normal numbers > 0, of an e4m3
 *                cache only; NULL: 1.  Another number: that head's codes are
 *                NaN, and SVW_DEV_BAD_INPUT.
 */
svw_status kv_append_norm(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                          int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
                          int64_t q_head_stride, void *q_out, svw_dtype dtype, int32_t n_q_heads, int32_t N,
                          const int32_t *cu_new, int64_t total_new, const int32_t *kv_len, const int32_t *positions,
                          const float *k_weight, const float *q_weight, float eps, const float *cos_sin,
                          int64_t max_pos, int32_t rot_dim, int32_t interleaved, const svw_paged_kv *cache,
                          svw_dtype cache_dtype, const float *k_scale, const float *v_scale, int32_t *status,
                          void *stream);

/*
 * kv_gather -- cached keys and values read back, packed: what a request keeps
 * when it leaves for another cache, or what a drafter reads of it.
 *
 * Output token t of request i (0 <= t < cu_out[i+1] - cu_out[i]) is its cached
 * token first[i] + t, in fp32 code x scale of its head (an e4m3 cache), rounded
 * once to out_dtype.
 *
 *   cache        of cache_dtype (any svw_dtype); head_dim <= 1024.
 *   k_scale, v_scale  as for kv_append_norm.
 *   cu_out       device int32 [N+1], cu_out[0] = 0, cu_out[N] = total_out.
 *   first        device int32 [N], >= 0; NULL: 0.
 *   k_out, v_out device [total_out, n_kv_heads, head_dim] of out_dtype (SVW_F32
 *                or SVW_BF16), contiguous; one of them may be NULL.
 *   status       SVW_DEV_BAD_INPUT when a token is in no request's valid range,
 *                lies before place 0 or beyond its block table, or its page is
 *                not one of the cache's (the token becomes NaN), or a scale is
 *                not a normal number > 0 (that head becomes NaN).
 * One kernel launch, no workspace.
 */
svw_status kv_gather(const svw_paged_kv *cache, svw_dtype cache_dtype, const float *k_scale, const float *v_scale,
                     int32_t N, const int32_t *cu_out, int64_t total_out, const int32_t *first, void *k_out,
                     void *v_out, svw_dtype out_dtype, int32_t *status, void *stream);

/*
 * paged_attention -- attention of each request's new tokens over its cached
 * keys (the new tokens' own ones included, as kv_append leaves them).
 *
 * New token t of request i (at place p = kv_len[i] - n_i + t) and query head
 * h see the keys j of head h / (n_q_heads / n_kv_heads) with
 *   0 <= j < kv_len[i],  causal: j <= p,  window > 0: j > p - window;
 *   out = sum_j softmax_j(scale q . k_j) v_j,  lse = log sum_j exp(scale q . k_j)
 * causal = 0: every new token sees the whole block (a diffusion drafter's).
 * A token that sees no key has out = 0 and lse = -inf.  kv_len[i] < n_i is
 * allowed: the tokens at negative places see nothing (causal).
 *
 *   q          device bf16 [total_new, n_q_heads, head_dim], strides of
 *              tokens and heads in elements; n_q_heads a multiple of
 *              n_kv_heads, at most 64 times it.
 *   cache      bf16; head_dim 64 or 128; page_size a power of two, 16 to 1024.
 *              What a token does not see (later tokens, places behind its
 *              window or beyond kv_len) may hold anything, NaN too; block-table
 *              entries of pages that no token sees are not looked at.
 *   scale      finite, > 0;  window >= 0, 0 unless causal.
 *   out        device bf16 [total_new, n_q_heads, head_dim], contiguous.
 *   lse        device float [total_new, n_q_heads], natural logarithm; may be NULL.
 *   workspace  device, 256-byte aligned, >= svw_paged_attention_workspace_size
 *              bytes; contents need not be initialised; not preserved.
 *   status     SVW_DEV_BAD_INPUT when a request's new-token range is invalid
 *              (nothing of it is written), its kv_len exceeds its block table
 *              (its out and lse become NaN) or a page that a token sees is not
 *              one of the cache's (that token's out and lse become NaN, those
 *              of tokens that do not see it are right).  After SVW_DEV_TIMEOUT a captured call is
 *              captured again before it is replayed.
 * q and the caches: 16-byte aligned, strides positive multiples of 8 elements
 * (those of dimensions of one do not count).
 * Scores and sums are fp32; the weights enter the second product in bf16.
 */
size_t svw_paged_attention_workspace_size(int64_t total_new, int32_t n_q_heads, int32_t n_kv_heads,
                                          int32_t head_dim);

svw_status paged_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, svw_dtype dtype,
                           int32_t n_q_heads, int32_t N, const int32_t *cu_new, int64_t total_new,
                           const int32_t *kv_len, const svw_paged_kv *cache, float scale, int32_t causal,
                           int32_t window, void *out, float *lse, int32_t *status, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * paged_attention_fp8 -- paged_attention over a cache of SVW_E4M3, as
 * kv_append_norm leaves it: with K and V the codes,
 *   s_j = scale k_scale[hk] q . K_j,  out = v_scale[hk] sum_j softmax_j(s) V_j,
 *   lse = log sum_j exp(s_j).
 *
 * Arguments, results and workspace size as for paged_attention, except:
 *   cache        codes of one byte; caches 16-byte aligned, strides positive
 *                multiples of 16.
 *   k_scale, v_scale  device float [n_kv_heads], normal numbers > 0; NULL: 1.
 *                Another number: the query heads of that key head become NaN
 *                (out and lse; v_scale: out), whether they see a key or not, and
 *                SVW_DEV_BAD_INPUT.
 * A query with a NaN or an infinity becomes NaN throughout, as one with scores
 * beyond 2.9 million in magnitude may (and does if its largest is).  Scores and sums are
 * fp32; a query enters its products as two e4m3 numbers under a scale of its
 * own, which is exact down to 2^-9 of its largest element (and within 2^-17 of
 * that one below); the weights enter the second product in fp16: within 2^-11 of
 * themselves down to 2^-21 of the largest, and within 2^-32 of that one below.
 * Beside the scores' and sums' fp32 roundings and its own to bf16, an output is so
 * within 2^-11 of sum_j w_j |v_j| and 2^-32 of the largest weight times sum_j |v_j|
 * (w normalised).
 */
svw_status paged_attention_fp8(const void *q, int64_t q_token_stride, int64_t q_head_stride, svw_dtype dtype,
                               int32_t n_q_heads, int32_t N, const int32_t *cu_new, int64_t total_new,
                               const int32_t *kv_len, const svw_paged_kv *cache, const float *k_scale,
                               const float *v_scale, float scale, int32_t causal, int32_t window, void *out,
                               float *lse, int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/*
 * spec_verify_noalloc -- spec_verify for callers that cannot allocate device
 * memory.  No counterpart on the pages: it exists only because some callers
 * have no allocator to hand over a workspace (a plain C serving loop, a
 * plug-in inside an engine whose memory pool is sized up front and which
 * forbids cudaMalloc -- a device-synchronising call -- mid-step, a thin launch
 * wrapper that only forwards tensors).
 *
 * Same arguments and results as spec_verify, minus the workspace: the library
 * keeps one fixed scratch area of SVW_NOALLOC_SCRATCH_BYTES per GPU (a
 * file-scope device array, resident for the life of the process on every GPU
 * that loads the library).  This call allocates nothing and frees nothing.
 *  - Batches whose svw_verify_workspace_size(...) exceeds the scratch return
 *    SVW_ERR_UNSUPPORTED without launching (e.g. N = 256 requests, 4096 draft
 *    rows at V = 151936 bf16 fit).
 *  - Argument checks run first and give spec_verify's codes; only a batch
 *    that passes them and needs more than the scratch gets SVW_ERR_UNSUPPORTED.
 *  - `stream` must belong to the current device (the scratch used is the
 *    current device's); otherwise SVW_ERR_INVALID_ARG, nothing launched.
 *  - The first call on each device looks the scratch's device address up
 *    (cudaGetSymbolAddress with that device current); make that first call
 *    before capturing the stream into a graph.
 *  - All calls share the scratch.  Calls whose kernels may overlap on the GPU
 *    (different streams without ordering, several host threads) race on it and
 *    corrupt each other's results; serialise them on one stream.
 */
#define SVW_NOALLOC_SCRATCH_BYTES (32u << 20)
svw_status spec_verify_noalloc(const void *target_logits, const void *draft_logits, svw_dtype dtype,
                               int32_t V, int32_t N, const int32_t *cu_draft,
                               int64_t total_draft_rows, int32_t max_len,
                               const int32_t *draft_tokens, float temperature, uint64_t seed,
                               int32_t *accept_len, int32_t *next_token, int32_t *status,
                               void *stream);

/*
 * svw_time_next_launch -- measurement hook, not part of the method.  Arms a
 * one-shot timer on the calling host thread: the next launch of the named
 * kernel made from this thread ("early_plan", "verify_stats",
 * "verify_finalize", "verify_early_cluster", "filter_rows", "filtered_finalize",
 * "opd_fast_kernel", "opd_fix_parts", "opd_fix_grad", "opd_exact_kernel",
 * "fused_finalize", "length_head_mma", "length_head_final", "adjust_lists",
 * "logits_adjust", "kv_append", "kv_append_norm", "kv_gather", "paged_attention", "paged_attention_fp8",
 * "attention_join") records
 * begin_event just before it and end_event just after it on the launch stream (cudaEvent_t handles passed as void*, owned
 * by the caller).  kernel = NULL disarms.  The library records nothing
 * unless armed.  Lets a benchmark time one kernel of a multi-kernel call with
 * CUDA events on the launch stream.
 */
svw_status svw_time_next_launch(const char *kernel, void *begin_event, void *end_event);

/*
 * Test hooks for the bounded waits, not part of the method ("failure
 * detection": a wait that runs out is reported, never a hang).
 *
 * svw_set_wait_limit -- the deadline, in SM clock cycles, of every bounded
 * wait in the library's kernels on the current device (default 4e9, about
 * 2 s).  cycles > 0, else SVW_ERR_INVALID_ARG.  Takes effect for kernels
 * launched after it returns.  A limit far below a copy's latency makes
 * healthy waits give up too; use it with svw_set_fault, at about 1e6 cycles,
 * so that only the injected wait runs out.
 *
 * svw_set_fault -- 0: none (default); 1: in the next calls until reset, CTA 0
 * of verify_stats (spec_verify) and cluster 0 of opd_fast_kernel
 * (opd_loss, spec_verify_opd) issue no bulk copy, so their first wait
 * runs out with nothing in flight, and so does CTA 0 of adjust_staged
 * (logits_adjust, a large batch out of place); every second worker of
 * paged_attention loads no values, so that the waits for its outputs run out
 * behind its scores, and in a call of few tokens one warp of the other workers
 * leaves before a part is marked, as if a wait of its own had run out.  The
 * call returns, its status word holds SVW_DEV_TIMEOUT, and the results of the
 * affected rows are void.  Other values: SVW_ERR_INVALID_ARG.  Host-side
 * state, shared by all threads.
 */
svw_status svw_set_wait_limit(int64_t cycles);
svw_status svw_set_fault(int32_t kind);

/* Human-readable name of a status code (static string). */
const char *svw_status_string(svw_status s);

/* Library ABI version: 100 * major + minor. */
int32_t svw_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SVW_H_ */
