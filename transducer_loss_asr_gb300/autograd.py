"""PyTorch autograd and torch.compile support for the TDT loss, cross attention and token log-probabilities.

The loss is registered as two custom ops over the split C ABI
(``tdt_loss_fwd`` / ``tdt_loss_bwd`` in include/tdt_loss.h):

* ``tdt_gb300::tdt_loss_forward`` -> (loss, workspace): node tables, alpha,
  beta and the arc fractions; the workspace (uint8) carries them to the
  backward op.
* ``tdt_gb300::tdt_loss_backward`` -> grad: the gradient pass only, scaled by
  the upstream gradient of the loss, so an arbitrary ``grad_output`` costs no
  extra pass over the gradient.

Both have fake implementations (shapes only), so the ops trace under
torch.compile(fullgraph=True) and pass torch.library.opcheck.  The pages'
layer gained the same properties in review: backward support, then fake
implementations, opcheck and compiled-vs-eager tests ("Add TDT loss kernel",
transformers PR #46048, thread on the kernel mapping).  The ops have CUDA
kernels only: called with CPU tensors they raise.
"""
from __future__ import annotations

from typing import List, Optional, Tuple

import torch
from torch import Tensor

REDUCTIONS = ("none", "sum", "mean", "mean_batch", "mean_volume")


def _align(v):
    return (v + 255) // 256 * 256


def workspace_nbytes(B, T, U1, n_dur):
    """Bytes of the split API's workspace for logits [B, T, U1, V+D].

    The same value as the C ABI's tdt_loss_workspace_size, written with
    integer arithmetic only so that it also holds for symbolic sizes under
    torch.compile: per anti-diagonal slot a node arc record of 2 * D arc
    probabilities, alpha and beta (8 bytes each: int32 exponent, float32
    mantissa) and a record of 2 + D arc fractions (float32); per node two
    log-sum-exps; per utterance likelihood, scale, flag and the lattice
    launch's start counter; every region 256-byte aligned.
    """
    ndiag = B * (T + U1 - 1) * U1
    nodes = B * T * U1
    rec_len = 2 * n_dur
    regions = (ndiag * 8 * rec_len, ndiag * 8, ndiag * 8, nodes * 4, nodes * 4,
               ndiag * 4 * (2 + n_dur), B * 8, B * 4, B * 4, B * 4)
    off = 0
    for r in regions:
        off = _align(off + r)
    return torch.sym_max(off, 256)


@torch.library.custom_op("tdt_gb300::tdt_loss_forward", mutates_args=(), device_types="cuda")
def tdt_loss_forward(logits: Tensor, labels: Tensor, logit_lengths: Tensor,
                     label_lengths: Tensor, durations: List[int], blank: int, sigma: float,
                     reduction: str) -> Tuple[Tensor, Tensor]:
    from . import binding

    B, T, U1, _ = logits.shape
    loss = torch.empty((B,) if reduction == "none" else (), dtype=torch.float32,
                       device=logits.device)
    # zero-filled: the kernels leave slots of nodes outside a lattice
    # unwritten, and an op's outputs must be a function of its inputs
    # (torch.compile and opcheck compare them)
    ws = torch.zeros(int(workspace_nbytes(B, T, U1, len(durations))), dtype=torch.uint8,
                     device=logits.device)
    loss, ws = binding.tdt_loss_fwd(logits, labels, logit_lengths, label_lengths, durations,
                                    blank, sigma, reduction, loss_out=loss, workspace=ws)
    return loss, ws


@tdt_loss_forward.register_fake
def _tdt_loss_forward_fake(logits, labels, logit_lengths, label_lengths, durations, blank, sigma,
                           reduction):
    B, T, U1, _ = logits.shape
    loss = logits.new_empty((B,) if reduction == "none" else (), dtype=torch.float32)
    ws = logits.new_empty((workspace_nbytes(B, T, U1, len(durations)),), dtype=torch.uint8)
    return loss, ws


@torch.library.custom_op("tdt_gb300::tdt_loss_backward", mutates_args=(), device_types="cuda")
def tdt_loss_backward(grad_loss: Tensor, logits: Tensor, labels: Tensor, logit_lengths: Tensor,
                      label_lengths: Tensor, workspace: Tensor, durations: List[int], blank: int,
                      sigma: float, reduction: str) -> Tensor:
    from . import binding

    g = grad_loss.to(torch.float32).contiguous()
    return binding.tdt_loss_bwd(logits, labels, logit_lengths, label_lengths, durations, blank,
                                workspace, grad_loss=g, sigma=sigma, reduction=reduction)


@tdt_loss_backward.register_fake
def _tdt_loss_backward_fake(grad_loss, logits, labels, logit_lengths, label_lengths, workspace,
                            durations, blank, sigma, reduction):
    return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)


def _setup_context(ctx, inputs, output):
    logits, labels, logit_lengths, label_lengths, durations, blank, sigma, reduction = inputs
    _, ws = output
    ctx.save_for_backward(logits, labels, logit_lengths, label_lengths, ws)
    ctx.args = (list(durations), blank, sigma, reduction)


def _backward(ctx, grad_loss, grad_ws):
    logits, labels, logit_lengths, label_lengths, ws = ctx.saved_tensors
    durations, blank, sigma, reduction = ctx.args
    grad = tdt_loss_backward(grad_loss, logits, labels, logit_lengths, label_lengths, ws,
                             durations, blank, sigma, reduction)
    return grad, None, None, None, None, None, None, None


tdt_loss_forward.register_autograd(_backward, setup_context=_setup_context)


def tdt_loss(logits: Tensor, labels: Tensor, logit_lengths: Tensor, label_lengths: Tensor,
             durations, blank: int, sigma: float = 0.0, reduction: str = "mean_volume") -> Tensor:
    """TDT loss of ``logits`` [B, T, U+1, V+D] (CUDA; float32/float16/bfloat16,
    may be a slice ``base[..., :V+D]``), differentiable w.r.t. ``logits``.

    labels: int64 [B, U] (padding -100); logit_lengths, label_lengths: int64
    [B]; durations: list of D distinct ints; blank in [0, V); sigma: logit
    under-normalisation; reduction: none | sum | mean | mean_batch |
    mean_volume.  Returns float32 [B] for "none", else a 0-dim tensor.
    """
    if reduction not in REDUCTIONS:
        raise ValueError("reduction must be one of %s" % (REDUCTIONS,))
    loss, _ = tdt_loss_forward(logits, labels, logit_lengths, label_lengths,
                               [int(d) for d in durations], int(blank), float(sigma), reduction)
    return loss


class TDTLoss(torch.nn.Module):
    """Stateless module form of :func:`tdt_loss` (same arguments)."""

    def forward(self, logits, labels, logit_lengths, label_lengths, durations, blank,
                sigma=0.0, reduction="mean_volume"):
        return tdt_loss(logits, labels, logit_lengths, label_lengths, durations, blank, sigma,
                        reduction)


# ---- cross attention ------------------------------------------------------------------------------


@torch.library.custom_op("tdt_gb300::cross_attention_forward", mutates_args=(), device_types="cuda")
def cross_attention_forward(q: Tensor, k: Tensor, v: Tensor, k_lens: Optional[Tensor],
                            q_lens: Optional[Tensor], windows: Optional[Tensor],
                            scale: float) -> Tuple[Tensor, Tensor]:
    from . import binding

    return binding.tdt_cross_attn_fwd(q, k, v, k_lens, q_lens, windows, scale)


@cross_attention_forward.register_fake
def _cross_attention_forward_fake(q, k, v, k_lens, q_lens, windows, scale):
    B, Lq, H, _ = q.shape
    return (torch.empty(q.shape, dtype=q.dtype, device=q.device),
            torch.empty((B, H, Lq), dtype=torch.float32, device=q.device))


@torch.library.custom_op("tdt_gb300::cross_attention_backward", mutates_args=(), device_types="cuda")
def cross_attention_backward(grad_out: Tensor, q: Tensor, k: Tensor, v: Tensor, out: Tensor,
                             lse: Tensor, k_lens: Optional[Tensor], q_lens: Optional[Tensor],
                             windows: Optional[Tensor],
                             scale: float) -> Tuple[Tensor, Tensor, Tensor]:
    from . import binding

    return binding.tdt_cross_attn_bwd(grad_out, q, k, v, out, lse, k_lens, q_lens, windows, scale)


@cross_attention_backward.register_fake
def _cross_attention_backward_fake(grad_out, q, k, v, out, lse, k_lens, q_lens, windows, scale):
    return tuple(torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))


def _cross_attention_setup(ctx, inputs, output):
    q, k, v, k_lens, q_lens, windows, scale = inputs
    out, lse = output
    ctx.save_for_backward(q, k, v, out, lse, k_lens, q_lens, windows)
    ctx.scale = scale
    ctx.mark_non_differentiable(lse)


def _cross_attention_backward(ctx, grad_out, grad_lse):
    q, k, v, out, lse, k_lens, q_lens, windows = ctx.saved_tensors
    dq, dk, dv = cross_attention_backward(grad_out, q, k, v, out, lse, k_lens, q_lens, windows,
                                          ctx.scale)
    return dq, dk, dv, None, None, None, None


cross_attention_forward.register_autograd(_cross_attention_backward,
                                          setup_context=_cross_attention_setup)


def cross_attention(q: Tensor, k: Tensor, v: Tensor, k_lens: Optional[Tensor] = None,
                    q_lens: Optional[Tensor] = None, windows: Optional[Tensor] = None,
                    scale: Optional[float] = None) -> Tensor:
    """Cross attention of label states ``q`` [B, Lq, H, D] to encoder frames ``k``, ``v``
    [B, Lk, Hkv, D] (CUDA; float32/float16/bfloat16; H a multiple of Hkv), differentiable w.r.t. q,
    k and v; the result is like q.

    k_lens, q_lens: int64 [B], frames and queries past them take no part; windows: int32 [B, Lq, 2],
    the frames [w0, w1) that each query sees; scale: 1 / sqrt(D) unless given.  A query that sees no
    frame gets zeros and no gradient.
    """
    scale = float(q.shape[-1]) ** -0.5 if scale is None else float(scale)
    return cross_attention_forward(q, k, v, k_lens, q_lens, windows, scale)[0]


class CrossAttention(torch.nn.Module):
    """Stateless module form of :func:`cross_attention` (same arguments)."""

    def forward(self, q, k, v, k_lens=None, q_lens=None, windows=None, scale=None):
        return cross_attention(q, k, v, k_lens, q_lens, windows, scale)


# ---- log-probabilities of given tokens ------------------------------------------------------------


@torch.library.custom_op("tdt_gb300::token_logprobs_forward", mutates_args=(), device_types="cuda")
def token_logprobs_forward(logits: Tensor, tokens: Tensor,
                           n_top: int) -> Tuple[Tensor, Tensor, Tensor, Tensor, Tensor]:
    from . import binding

    r = binding.tdt_token_logprobs_fwd(logits, tokens, n_top)
    if n_top:
        return tuple(r)
    N = logits.shape[0]
    return (*r[:3], logits.new_empty((N, 0), dtype=torch.int32),
            logits.new_empty((N, 0), dtype=torch.float32))


@token_logprobs_forward.register_fake
def _token_logprobs_forward_fake(logits, tokens, n_top):
    N, f = logits.shape[0], torch.float32
    return (logits.new_empty((N,), dtype=f), logits.new_empty((N,), dtype=f),
            logits.new_empty((N, 2), dtype=f), logits.new_empty((N, n_top), dtype=torch.int32),
            logits.new_empty((N, n_top), dtype=f))


@torch.library.custom_op("tdt_gb300::token_logprobs_backward", mutates_args=(), device_types="cuda")
def token_logprobs_backward(grad_logprobs: Optional[Tensor], grad_entropy: Optional[Tensor],
                            grad_top: Optional[Tensor], logits: Tensor, tokens: Tensor, entropy: Tensor,
                            stats: Tensor, top_tokens: Tensor) -> Tensor:
    from . import binding

    a, b, c = (None if g is None else g.contiguous() for g in (grad_logprobs, grad_entropy, grad_top))
    r = binding.TokenLogprobs(entropy, entropy, stats, top_tokens)
    return binding.tdt_token_logprobs_bwd(logits, tokens, r, a, b, c)


@token_logprobs_backward.register_fake
def _token_logprobs_backward_fake(grad_logprobs, grad_entropy, grad_top, logits, tokens, entropy, stats,
                                  top_tokens):
    return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)


def _token_logprobs_setup(ctx, inputs, output):
    logits, tokens, n_top = inputs
    _, entropy, stats, top_tokens, _ = output
    ctx.save_for_backward(logits, tokens, entropy, stats, top_tokens)
    ctx.n_top = n_top
    ctx.mark_non_differentiable(stats, top_tokens)
    ctx.set_materialize_grads(False)


def _token_logprobs_backward(ctx, grad_logprobs, grad_entropy, grad_stats, grad_tokens, grad_top):
    if grad_logprobs is None and grad_entropy is None and grad_top is None:
        return None, None, None
    grad = token_logprobs_backward(grad_logprobs, grad_entropy, grad_top if ctx.n_top else None,
                                   *ctx.saved_tensors)
    return grad, None, None


token_logprobs_forward.register_autograd(_token_logprobs_backward, setup_context=_token_logprobs_setup)


def token_logprobs(logits: Tensor, tokens: Tensor,
                   n_top: int = 0) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    """(logprobs, entropy, top_tokens, top_logprobs) of ``tokens`` [...] under ``logits`` [..., V] (CUDA;
    float32/float16/bfloat16; may be a slice ``base[..., :V]``): the log-probability of each token, the
    entropy of its row, and the n_top most probable tokens ([..., n_top], int32) with theirs.
    Differentiable w.r.t. logits through logprobs, entropy and top_logprobs.

    tokens: int64; a negative one is padding (-100): its row takes no part, and its results are 0
    (alternatives -1 and -inf).  -sum(logprobs) is the cross entropy of the labels.
    """
    V, shape = logits.shape[-1], tokens.shape
    if logits.shape[:-1] != shape:
        raise ValueError("tokens must be of shape %s" % (tuple(logits.shape[:-1]),))
    lp, entropy, _, top, top_lp = token_logprobs_forward(
        logits.reshape(-1, V), tokens.reshape(-1).contiguous(), int(n_top))
    return lp.view(shape), entropy.view(shape), top.view(*shape, n_top), top_lp.view(*shape, n_top)


class TokenLogprobs(torch.nn.Module):
    """Stateless module form of :func:`token_logprobs` (same arguments)."""

    def forward(self, logits, tokens, n_top=0):
        return token_logprobs(logits, tokens, n_top)
