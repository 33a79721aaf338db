/*
 * tdt_decoder.h -- C ABI of the attention-decoder operators of the GB300
 * (sm_103a) transducer library: cross attention of label states to encoder
 * frames (forward and backward), drawing tokens from logits, the label
 * states' own paged cache with the causal attention that reads it, and
 * log-probabilities of given tokens with their gradient.
 *
 * They stand next to the TDT loss (tdt_loss.h) in a hybrid transducer /
 * attention model: label states read the encoder's frames, in training
 * (tdt_cross_attn_fwd, tdt_cross_attn_bwd) and while decoding or rescoring a
 * transducer's hypotheses (tdt_cross_attn_fwd on a few rows), and tokens are
 * drawn at random instead of by argmax (tdt_sample).  While decoding, the label
 * states of a hypothesis read each other through a paged cache
 * (tdt_cache_write, tdt_paged_attn); hypotheses are scored, and the decoder
 * trained, by tdt_token_logprobs_fwd, _bwd and _fwd_bwd.
 *
 * Conventions are those of tdt_loss.h: the caller owns every pointer,
 * `sizes` and `strides` are host arrays, tensors are device memory, calls are
 * asynchronous on `stream` (a cudaStream_t, NULL: the legacy default stream)
 * and never synchronise, a negative TDT_ERR_* status is returned before
 * anything is enqueued when an argument is invalid, and what only the device
 * can see never traps.
 */
#ifndef TDT_DECODER_H
#define TDT_DECODER_H

#include "tdt_loss.h"

#ifdef __cplusplus
extern "C" {
#endif

/* head layout: H must be a positive multiple of Hkv, 1 <= D <= 256 */
#define TDT_ERR_BAD_HEADS (-14)
/* scale must be finite and positive */
#define TDT_ERR_BAD_SCALE (-15)
/* a sampling setting is out of range */
#define TDT_ERR_BAD_SAMPLING (-16)

/*
 * Cross attention.  Query i of utterance b and head h sees the frames
 *   R(b,i) = { j : max(0, w0) <= j < min(k_lens[b], w1) },  (w0, w1) = windows[b][i],
 * none when i >= q_lens[b]; key/value head c = h / (H / Hkv) serves the
 * H / Hkv query heads of its group.
 *   s_j = scale q . k_j      lse = ln sum_{j in R} exp(s_j)
 *   out = sum_{j in R} exp(s_j - lse) v_j
 * A query that sees no frame gets out = 0, lse = -inf and no gradient.
 *
 *   sizes    {B, Lq, Lk, H, Hkv, D}; B, Lq, Lk >= 0 (Lk = 0: no query sees a
 *            frame), Lq, Lk < 2^30, B * H < 2^31 / max(1, Lq / 32).
 *   strides  element strides of (batch, position, head) of each tensor, the
 *            head's D elements being contiguous: q[B, Lq, H, D],
 *            k[B, Lk, Hkv, D], v[B, Lk, Hkv, D], out[B, Lq, H, D] for the
 *            forward call; then grad_out[B, Lq, H, D], dq[B, Lq, H, D],
 *            dk, dv [B, Lk, Hkv, D] for the backward call.  Inputs may have
 *            any strides >= 0 (0: broadcast; slices of a fused projection);
 *            no two elements of an output may share an address.
 *   dtype    TDT_DTYPE_* of every tensor but lse.  Sums, the softmax and lse
 *            are held in float32.
 *   k_lens   device int64 [B] or NULL (all Lk).   q_lens: int64 [B] or NULL
 *            (all Lq), e.g. label_lens + 1.  Frames at or past k_lens[b] and
 *            queries at or past q_lens[b] may hold anything, NaN included;
 *            frames before k_lens[b] that a query's window leaves out, and
 *            queries before q_lens[b] whose window is empty, are to be finite,
 *            and so their products (their weight is 0, and is multiplied).  A length outside [0, Lk] or [0, Lq] gives that
 *            utterance NaN outputs and zero gradients.
 *   windows  device int32 [B, Lq, 2] contiguous or NULL, e.g. around the
 *            frames that tdt_greedy_decode emits tokens at.
 *   scale    finite and > 0, usually 1 / sqrt(D).
 *   lse      device float32 [B, H, Lq] contiguous (natural logarithm); may be
 *            NULL in the forward call when no gradient is wanted.
 *   workspace  device, 256-byte aligned, at least
 *            tdt_cross_attn_workspace_size(sizes, dtype, backward) bytes; may be
 *            NULL when that is 0.  Not used by anything else until the
 *            stream has passed the call.
 * Results do not depend on what else runs: every sum has a fixed order.
 */
size_t tdt_cross_attn_workspace_size(const int64_t sizes[6], int dtype, int backward);

int tdt_cross_attn_fwd(const void *q, const void *k, const void *v, const int64_t sizes[6],
                       const int64_t strides[12], int dtype, const int64_t *k_lens,
                       const int64_t *q_lens, const int32_t *windows, double scale, void *out,
                       float *lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gradients of sum(grad_out * out): with p_ij = exp(s_ij - lse_i) and
 * delta_i = grad_out_i . out_i,
 *   ds_ij = p_ij (grad_out_i . v_j - delta_i),
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,
 *   dv_j = sum_i p_ij grad_out_i,
 * the last two summed over the query heads of the group.  out and lse are the
 * forward call's; every other argument equals the forward call's.
 *   strides  24 values: q, k, v, out, grad_out, dq, dk, dv (three each).
 * Every element of dq, dk and dv is written (rows that take no part: 0).
 */
int tdt_cross_attn_bwd(const void *grad_out, const void *q, const void *k, const void *v,
                       const void *out, const float *lse, const int64_t sizes[6],
                       const int64_t strides[24], int dtype, const int64_t *k_lens,
                       const int64_t *q_lens, const int32_t *windows, double scale, void *dq,
                       void *dk, void *dv, void *workspace, size_t workspace_bytes,
                       void *stream);

/*
 * Draws a token of each row of logits from a given uniform number.
 *
 * With x the row, X its maximum and T the temperature, token i weighs
 *   w_i = rint(2^31 * 2^((x_i - X) * (log2(e) / T)))        (a whole number)
 * and the tokens are ordered by falling x_i, equal ones by rising index.  Of
 * that order a prefix stays, at least its first token:
 *   top_k  (0 or >= V: off)  the first top_k tokens;
 *   top_p  (1: off)          of those, the tokens with less than
 *                            floor(sum w * top_p) weight before them;
 *   min_p  (0: off)          the tokens with w_i >= ceil(2^31 min_p).
 * With W the weight that stays, the token drawn is the first, in the order of
 * the vocabulary, at which the running sum of the weights that stay exceeds
 * floor(W * u).  top_p and u are taken to 24 bits.  The weights are whole
 * numbers, so every sum is exact and the draw does not depend on the order of
 * additions: the same inputs give the same token on any launch shape.
 * T = 0 draws the first token of the order.  logprob = log-probability of the
 * token among those that stay.
 *
 *   logits     device [N, V] of `dtype`, row n at logits + n * row_stride
 *              elements, elements contiguous: a slice [..., :V] of a wider
 *              tensor needs no copy; rows need no alignment beyond the
 *              element's.  -inf and NaN entries are never drawn; a row of
 *              nothing else gives token -1 and logprob NaN.
 *   sizes      {N, V}; N >= 0, 1 <= V <= 2^24.
 *   uniforms   device float32 [N], in [0, 1) (others are clamped).
 *   temperatures, top_ps, min_ps  device float32 [N]; top_ks device int32
 *              [N]; each may be NULL: the call's own value then holds for all
 *              rows (temperature finite and >= 0, 0 <= top_p, min_p <= 1,
 *              top_k >= 0).  A row's own value out of range gives token -1
 *              and logprob NaN.
 *   tokens     device int32 [N].     logprobs  device float32 [N] or NULL.
 */
int tdt_sample(const void *logits, const int64_t sizes[2], int64_t row_stride, int dtype,
               const float *uniforms, const float *temperatures, const int32_t *top_ks,
               const float *top_ps, const float *min_ps, double temperature, int64_t top_k,
               double top_p, double min_p, int32_t *tokens, float *logprobs, void *stream);

/* ------------------------------------------------------------------------
 * A paged cache of label states' keys and values.
 *
 * Position p of utterance b lies in page page_table[b][p / page_size], place
 * p % page_size.  Pages are shared by utterances and hypotheses as their
 * tables say; nothing here owns or counts them.
 */

/* of cache pages only: 8-bit floats (4 exponent, 3 mantissa bits, no infinities) */
#define TDT_DTYPE_E4M3 3
/* n_pages, page_size, or the page table is out of range */
#define TDT_ERR_BAD_PAGES (-17)
/* n_top must be in [0, min(V, 64)] */
#define TDT_ERR_BAD_TOP (-18)

/*
 *   k_pages, v_pages  device [n_pages, page_size, n_heads, head_dim] of
 *               `dtype`: the tensors' own type, or TDT_DTYPE_E4M3.
 *   k_scales, v_scales  device uint8 [n_pages, page_size, n_heads], with
 *               TDT_DTYPE_E4M3 only (else NULL): a row of head_dim elements
 *               stands for e4m3 * 2^(byte - 127); byte 255: for NaN.
 *               (Rounding may take what is past 1.9375 * 2^127 to infinity.)
 *   n_pages     in [1, 2^31).   page_size  a power of two, at most 2^16.
 *   n_heads >= 1, 1 <= head_dim <= 256.
 *   strides     elements, of (page, place, head) of k_pages, v_pages,
 *               k_scales, v_scales, all >= 0; a row's elements are contiguous.
 *               No two rows of a cache that is written may share an address.
 */
typedef struct tdt_paged_cache {
  void *k_pages, *v_pages;
  uint8_t *k_scales, *v_scales;
  int64_t n_pages, page_size, n_heads, head_dim;
  int64_t strides[12];
  int32_t dtype;
} tdt_paged_cache;

/*
 * Writes rows of k and v into their pages.  Row i < q_lens[b] of utterance b
 * is position kv_lens[b] - q_lens[b] + i: kv_lens counts the new rows too, so
 * the same lengths serve tdt_paged_attn afterwards.  With TDT_DTYPE_E4M3 a
 * row x is quantised as it is written: with e the least whole number in
 * [-117, 120] that keeps max |x| <= 448 * 2^e, it is stored as the e4m3
 * nearest to x * 2^-e (ties to even) and the byte e + 127.  A power of two
 * costs a floating format no precision, and reading back is exact.  A row
 * with a NaN or an infinity gets byte 255.
 *
 *   sizes    {B, L, max_pages}; k, v [B, L, n_heads, head_dim].
 *   strides  elements, of (batch, position, head) of k, then v; >= 0.
 *   dtype    TDT_DTYPE_F32, F16 or BF16, of k and v; pages that are not
 *            TDT_DTYPE_E4M3 have the same.
 *   page_table  device int32 [B, max_pages], row b at b * table_stride.
 *   kv_lens  device int64 [B].   q_lens  device int64 [B] or NULL (all L).
 * Nothing is written for an utterance whose q_lens is outside [0, L] or
 * whose kv_lens is outside [q_lens, max_pages * page_size], nor for rows
 * whose page is outside [0, n_pages).  Rows at or past q_lens[b] are not
 * read, and places that no row goes to keep what they hold.  Where two rows of
 * a call go to one place (hypotheses that share the page), their values must
 * be the same.
 */
int tdt_cache_write(const void *k, const void *v, const int64_t sizes[3], const int64_t strides[6],
                    int dtype, const tdt_paged_cache *cache, const int32_t *page_table,
                    int64_t table_stride, const int64_t *kv_lens, const int64_t *q_lens,
                    void *stream);

/*
 * Reads back what tdt_cache_write of the same arguments wrote: rows i <
 * q_lens[b], positions kv_lens[b] - q_lens[b] + i (q_lens = kv_lens: whole
 * utterances), rounded to `dtype` once.  Pages of any type give any of the
 * three types.  Rows at or past q_lens[b] are 0; rows of an utterance with
 * lengths out of range, or of a page outside [0, n_pages), are NaN.
 */
int tdt_cache_read(const tdt_paged_cache *cache, const int32_t *page_table, int64_t table_stride,
                   const int64_t *kv_lens, const int64_t *q_lens, const int64_t sizes[3],
                   const int64_t strides[6], int dtype, void *k, void *v, void *stream);

/*
 * Causal attention of new label states over their cache, which holds their
 * own keys and values already.  Query i < q_lens[b] of utterance b is at
 * position kv_lens[b] - q_lens[b] + i and sees the positions up to its own;
 * head c = h / (H / n_heads) of the cache serves query head h:
 *   s_j = scale q . k_j      lse = ln sum exp(s_j)      out = sum exp(s_j - lse) v_j
 * One query an utterance is a decoding step, more are a prompt or a
 * hypothesis to rescore.  Queries at or past q_lens[b] get out = 0, lse = -inf.
 *
 *   sizes    {B, Lq, H, max_pages}; Lq < 2^30, max_pages * page_size < 2^30.
 *   strides  elements, of (batch, position, head) of q[B, Lq, H, head_dim],
 *            then out; inputs >= 0; no two elements of out may share an address.
 *   dtype    of q and out; pages that are not TDT_DTYPE_E4M3 have the same.
 *            Scores, the softmax, sums and lse are held in float32; values
 *            of e4m3 pages enter as they are, without a rounding in between
 *            (but with float16 queries they may end at 65504).  Weights of
 *            16-bit calls are rounded to 16 bits; with few queries over e4m3
 *            pages to float16, times the value row's power of two relative to
 *            the utterance's largest: rows more than 2^21 smaller than that
 *            one lose bits of their weights, and more than 2^31 smaller all.
 *   kv_lens, q_lens, page_table  as in tdt_cache_write.  Lengths out of range
 *            give that utterance NaN; a page outside [0, n_pages) gives NaN to
 *            the queries that see it, and may to the utterance's others.
 *            Places past kv_lens[b] may hold anything, NaN included; positions
 *            before it are to be finite, and so are scores and 2^15 times the
 *            sums of values (weights are divided by their sum at the end, and
 *            may be that large until then).
 *   lse      device float32 [B, H, Lq] contiguous, or NULL.
 *   workspace  device, 256-byte aligned, at least
 *            tdt_paged_attn_workspace_size(sizes, dtype, cache) bytes; may be
 *            NULL when that is 0.  Not used by anything else until the stream
 *            has passed the call.  Many queries over e4m3 pages, and what the
 *            paged kernels do not take (float32 with many queries, heads over
 *            128, rows that no 16-byte access fits, pages of under 8 places), need
 *            room for B * max_pages * page_size dense rows of k and v of `dtype`:
 *            a table that is no wider than needed keeps it small.
 */
size_t tdt_paged_attn_workspace_size(const int64_t sizes[4], int dtype, const tdt_paged_cache *cache);

int tdt_paged_attn(const void *q, const int64_t sizes[4], const int64_t strides[6], int dtype,
                   const tdt_paged_cache *cache, const int32_t *page_table, int64_t table_stride,
                   const int64_t *kv_lens, const int64_t *q_lens, double scale, void *out,
                   float *lse, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Log-probabilities of given tokens.
 *
 * With x a row of logits, p = softmax(x) and t its token:
 *   logprob = ln p_t      entropy = -sum_i p_i ln p_i  (0 ln 0 = 0)
 * and the alternatives are the n_top most probable tokens, by falling x,
 * equal ones by rising index, each with its log-probability.  Entries of
 * -inf (tokens that are not allowed) have p = 0.
 *
 *   logits   device [N, V] of `dtype`, row n at logits + n * row stride,
 *            elements contiguous; rows need no alignment beyond the element's.
 *   sizes    {N, V, n_top}; 0 <= N < 2^27, 1 <= V <= 2^24,
 *            0 <= n_top <= min(V, 64).
 *   tokens   device int64 [N].  A negative one (the labels' padding of -100)
 *            leaves its row out: the row is not read and may hold anything;
 *            logprob, entropy and stats are 0, the alternatives -1 and -inf,
 *            the gradient 0.  One >= V gives NaN (alternatives -1) and a
 *            gradient of 0.
 *   logprobs device float32 [N].   entropy  device float32 [N] or NULL.
 *   stats    device float32 [N, 2] or NULL: the row's maximum m, and
 *            ln sum exp(x - m); their sum is ln sum exp(x).
 *   top_tokens, top_logprobs  device int32, float32 [N, n_top]; NULL if n_top
 *            is 0.  Alternatives that are not allowed have logprob -inf.
 * A row that holds NaN or +inf, or nothing but -inf, gives NaN (alternatives
 * -1 and NaN).  Results do not depend on what else runs.
 */
int tdt_token_logprobs_fwd(const void *logits, const int64_t sizes[3], int64_t row_stride, int dtype,
                           const int64_t *tokens, float *logprobs, float *entropy, float *stats,
                           int32_t *top_tokens, float *top_logprobs, void *stream);

/*
 * The gradient of sum_n a_n logprob_n + b_n entropy_n + sum_j c_nj top_logprob_nj:
 *   dx_i = a [i = t] + sum_j c_j [i = top_j] - p_i (a + sum_j c_j) - b p_i (ln p_i + entropy)
 *   strides     {row stride of logits, of grad_out}; the latter >= V.
 *   entropy, stats, top_tokens  the forward call's; entropy may be NULL
 *               without grad_entropy, top_tokens without grad_top.
 *   grad_logprobs, grad_entropy  a and b, device float32 [N], or NULL (0).
 *   grad_top    c, device float32 [N, n_top], or NULL (0).
 *   grad_out    device [N, V] of `dtype`; may be `logits` with the same stride
 *               (the gradient then replaces them), and may not overlap it in
 *               any other way (TDT_ERR_BAD_ALIASING).
 * Every element of grad_out's rows is written.  Rows of NaN results get a
 * gradient of NaN, but for tokens >= V.
 */
int tdt_token_logprobs_bwd(const void *logits, const int64_t sizes[3], const int64_t strides[2],
                           int dtype, const int64_t *tokens, const float *entropy,
                           const float *stats, const int32_t *top_tokens,
                           const float *grad_logprobs, const float *grad_entropy,
                           const float *grad_top, void *grad_out, void *stream);

/*
 * Both in one call, where a and b are known beforehand (cross entropy with its
 * label weights): the logits are read from memory once.  Arguments as above.
 */
int tdt_token_logprobs_fwd_bwd(const void *logits, const int64_t sizes[3], const int64_t strides[2],
                               int dtype, const int64_t *tokens, const float *grad_logprobs,
                               const float *grad_entropy, float *logprobs, float *entropy,
                               float *stats, int32_t *top_tokens, float *top_logprobs,
                               void *grad_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TDT_DECODER_H */
