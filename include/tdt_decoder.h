/*
 * tdt_decoder.h -- C ABI of the attention-decoder operators of the GB300
 * (sm_103a) transducer library: cross attention of label states to encoder
 * frames (forward and backward), and drawing tokens from logits.
 *
 * They stand next to the TDT loss (tdt_loss.h) in a hybrid transducer /
 * attention model: label states read the encoder's frames, in training
 * (tdt_cross_attn_fwd, tdt_cross_attn_bwd) and while decoding or rescoring a
 * transducer's hypotheses (tdt_cross_attn_fwd on a few rows), and tokens are
 * drawn at random instead of by argmax (tdt_sample).
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

#ifdef __cplusplus
}
#endif

#endif /* TDT_DECODER_H */
