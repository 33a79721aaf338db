"""ctypes binding of libtdt_loss.so (include/tdt_loss.h, include/tdt_decoder.h).

Argument marshalling only: sizes, strides, dtype codes, raw pointers and the
current CUDA stream go to the C ABI; every step of the loss runs in the
library's kernels.  PyTorch is used for device memory and streams.  There is
no fallback: if the library is missing, importing this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtdt_loss.so")

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
REDUCTIONS = {"none": 0, "sum": 1, "mean": 2, "mean_batch": 3, "mean_volume": 4}

TDT_OK = 0


class TDTError(RuntimeError):
    """A TDT_ERR_* status returned by the library."""

    def __init__(self, status: int, text: str):
        super().__init__("tdt_loss status %d: %s" % (status, text))
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libtdt_loss.so is not built (%s); run `python -m transducer_loss_asr_gb300.build` "
            "or __graft_entry__.build()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    I = ctypes.c_int
    common = [P, P, P, I, P, P, P, P, I, I, ctypes.c_double, I, P, P]
    lib.tdt_loss_fwd_bwd.restype = I
    lib.tdt_loss_fwd_bwd.argtypes = common + [P]
    lib.tdt_loss_fwd_bwd_ws.restype = I
    lib.tdt_loss_fwd_bwd_ws.argtypes = common + [P, ctypes.c_size_t, P]
    lib.tdt_loss_fwd_bwd_noalloc.restype = I
    lib.tdt_loss_fwd_bwd_noalloc.argtypes = common + [P]
    lib.tdt_rnnt_loss_fwd_bwd.restype = I
    lib.tdt_rnnt_loss_fwd_bwd.argtypes = [P, P, P, I, P, P, P, I, ctypes.c_double, I, P, P, P]
    lib.tdt_greedy_decode.restype = I
    lib.tdt_greedy_decode.argtypes = [P, P, P, I, P, P, I, I, I, P, P, P, P, P]
    lib.tdt_loss_fwd.restype = I
    lib.tdt_loss_fwd.argtypes = common[:-1] + [P, ctypes.c_size_t, P]
    lib.tdt_loss_bwd.restype = I
    lib.tdt_loss_bwd.argtypes = common[:-2] + [P, P, P, ctypes.c_size_t, P]
    lib.tdt_loss_workspace_size.restype = ctypes.c_size_t
    lib.tdt_loss_workspace_size.argtypes = [P, I]
    lib.tdt_status_string.restype = ctypes.c_char_p
    lib.tdt_status_string.argtypes = [I]
    lib.tdt_loss_version.restype = I
    lib.tdt_loss_version.argtypes = []
    lib.tdt_loss_set_lattice_bands.restype = I
    lib.tdt_loss_set_lattice_bands.argtypes = [I]
    lib.tdt_loss_set_lattice_exchange.restype = I
    lib.tdt_loss_set_lattice_exchange.argtypes = [I]
    lib.tdt_loss_test_set_halo_fault.restype = ctypes.c_longlong
    lib.tdt_loss_test_set_halo_fault.argtypes = [ctypes.c_longlong, ctypes.c_longlong]
    lib.tdt_loss_timing_enable.restype = None
    lib.tdt_loss_timing_enable.argtypes = [I]
    lib.tdt_loss_timing_read.restype = I
    lib.tdt_loss_timing_read.argtypes = [P, P, P, I, I]
    lib.tdt_cross_attn_workspace_size.restype = ctypes.c_size_t
    lib.tdt_cross_attn_workspace_size.argtypes = [P, I, I]
    lib.tdt_cross_attn_fwd.restype = I
    lib.tdt_cross_attn_fwd.argtypes = [P, P, P, P, P, I, P, P, P, ctypes.c_double, P, P, P,
                                       ctypes.c_size_t, P]
    lib.tdt_cross_attn_bwd.restype = I
    lib.tdt_cross_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, I, P, P, P, ctypes.c_double, P, P,
                                       P, P, ctypes.c_size_t, P]
    lib.tdt_sample.restype = I
    lib.tdt_sample.argtypes = [P, P, ctypes.c_int64, I, P, P, P, P, P, ctypes.c_double,
                               ctypes.c_int64, ctypes.c_double, ctypes.c_double, P, P, P]
    I64 = ctypes.c_int64
    lib.tdt_cache_write.restype = I
    lib.tdt_cache_write.argtypes = [P, P, P, P, I, P, P, I64, P, P, P]
    lib.tdt_cache_read.restype = I
    lib.tdt_cache_read.argtypes = [P, P, I64, P, P, P, P, I, P, P, P]
    lib.tdt_paged_attn_workspace_size.restype = ctypes.c_size_t
    lib.tdt_paged_attn_workspace_size.argtypes = [P, I, P]
    lib.tdt_paged_attn.restype = I
    lib.tdt_paged_attn.argtypes = [P, P, P, I, P, P, I64, P, P, ctypes.c_double, P, P, P,
                                   ctypes.c_size_t, P]
    lib.tdt_token_logprobs_fwd.restype = I
    lib.tdt_token_logprobs_fwd.argtypes = [P, P, I64, I, P, P, P, P, P, P, P]
    lib.tdt_token_logprobs_bwd.restype = I
    lib.tdt_token_logprobs_bwd.argtypes = [P, P, P, I, P, P, P, P, P, P, P, P, P]
    lib.tdt_token_logprobs_fwd_bwd.restype = I
    lib.tdt_token_logprobs_fwd_bwd.argtypes = [P, P, P, I, P, P, P, P, P, P, P, P, P, P]
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.tdt_status_string(int(status)).decode()


def _check(status: int):
    if status != TDT_OK:
        raise TDTError(status, status_string(status))


def _i64(vals):
    return (ctypes.c_int64 * 4)(*[int(v) for v in vals])


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _addr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def workspace_size(sizes, n_dur: int) -> int:
    return int(lib.tdt_loss_workspace_size(_i64(sizes), int(n_dur)))


def _marshal(logits, labels, logit_lens, label_lens, durations, blank, sigma, reduction,
             loss_out, grad_out, compute_grad, with_loss=True):
    if logits.dim() != 4:
        raise ValueError("logits must be [B, T, U+1, V+D]")
    if logits.dtype not in DTYPES:
        raise TypeError("logits dtype must be float32, float16 or bfloat16")
    B = logits.shape[0]
    dev = logits.device
    if loss_out is None and with_loss:
        loss_out = torch.empty(B if reduction == "none" else 1, dtype=torch.float32, device=dev)
    if compute_grad and grad_out is None:
        grad_out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    if grad_out is not None and (not grad_out.is_contiguous() or grad_out.dtype != logits.dtype
                                 or tuple(grad_out.shape) != tuple(logits.shape)):
        raise ValueError("grad_out must be contiguous with the logits' shape and dtype")
    durs = (ctypes.c_int32 * len(durations))(*[int(d) for d in durations])
    args = [
        _ptr(logits), _i64(logits.shape), _i64(logits.stride()), DTYPES[logits.dtype],
        _ptr(labels) if labels is not None and labels.numel() > 0 else None,
        _ptr(logit_lens), _ptr(label_lens), durs, len(durations), int(blank), float(sigma),
        REDUCTIONS[reduction], _ptr(loss_out), _ptr(grad_out),
    ]
    for name, t in (("labels", labels), ("logit_lens", logit_lens), ("label_lens", label_lens)):
        if t is not None and (t.dtype != torch.int64 or not t.is_contiguous() or t.device != dev):
            raise ValueError("%s must be a contiguous int64 tensor on %s" % (name, dev))
    return args, loss_out, grad_out


def tdt_loss_fwd_bwd(logits, labels, logit_lens, label_lens, durations, blank, sigma=0.0,
                     reduction="mean_volume", loss_out=None, grad_out=None, compute_grad=True):
    """TDT loss and its gradient in one call on the current CUDA stream.

    Returns (loss, grad): loss float32 [B] ("none") or [1]; grad with the
    logits' shape and dtype (None when compute_grad is False and no grad_out
    is given).  ``logits`` may be a strided view such as ``base[..., :V+D]``.
    """
    args, loss_out, grad_out = _marshal(logits, labels, logit_lens, label_lens, durations,
                                        blank, sigma, reduction, loss_out, grad_out,
                                        compute_grad)
    with torch.cuda.device(logits.device):
        _check(lib.tdt_loss_fwd_bwd(*args, _stream_handle(logits.device)))
    return loss_out, grad_out


def tdt_rnnt_loss_fwd_bwd(logits, labels, logit_lens, label_lens, blank, sigma=0.0,
                          reduction="mean_volume", loss_out=None, grad_out=None,
                          compute_grad=True):
    """Plain RNN-T loss (no duration head) and its gradient on the current
    CUDA stream: logits [B, T, U+1, V]; other arguments as tdt_loss_fwd_bwd
    without durations.  Returns (loss, grad)."""
    args, loss_out, grad_out = _marshal(logits, labels, logit_lens, label_lens, [0], blank,
                                        sigma, reduction, loss_out, grad_out, compute_grad)
    # drop the durations pointer and count of the TDT argument list
    rargs = args[:7] + args[9:]
    with torch.cuda.device(logits.device):
        _check(lib.tdt_rnnt_loss_fwd_bwd(*rargs, _stream_handle(logits.device)))
    return loss_out, grad_out


def tdt_greedy_decode(logits, logit_lens, durations, blank, max_symbols=10):
    """Greedy TDT decoding of joint outputs ``logits`` [B, T, U+1, V+D] on the
    current CUDA stream.  Returns (n [B], tokens, frames, token_durations
    [B, U+1]) as int32 CUDA tensors, -1 past n[b]."""
    if logits.dim() != 4:
        raise ValueError("logits must be [B, T, U+1, V+D]")
    if logits.dtype not in DTYPES:
        raise TypeError("logits dtype must be float32, float16 or bfloat16")
    if logit_lens.dtype != torch.int64 or logit_lens.device != logits.device:
        raise ValueError("logit_lens must be an int64 tensor on %s" % logits.device)
    B, _, U1, _ = logits.shape
    dev = logits.device
    n = torch.empty(B, dtype=torch.int32, device=dev)
    tok, frm, dur = (torch.empty(B, U1, dtype=torch.int32, device=dev) for _ in range(3))
    durs = (ctypes.c_int32 * len(durations))(*[int(d) for d in durations])
    with torch.cuda.device(dev):
        _check(lib.tdt_greedy_decode(
            _ptr(logits), _i64(logits.shape), _i64(logits.stride()), DTYPES[logits.dtype],
            _ptr(logit_lens.contiguous()), durs, len(durations), int(blank), int(max_symbols),
            _ptr(n), _ptr(tok), _ptr(frm), _ptr(dur), _stream_handle(dev)))
    return n, tok, frm, dur


def _check_workspace(workspace, dev):
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % dev)


def tdt_loss_fwd_bwd_ws(logits, labels, logit_lens, label_lens, durations, blank, workspace,
                        sigma=0.0, reduction="mean_volume", loss_out=None, grad_out=None,
                        compute_grad=True):
    """As tdt_loss_fwd_bwd with a caller-owned uint8 CUDA workspace tensor."""
    _check_workspace(workspace, logits.device)
    args, loss_out, grad_out = _marshal(logits, labels, logit_lens, label_lens, durations,
                                        blank, sigma, reduction, loss_out, grad_out,
                                        compute_grad)
    with torch.cuda.device(logits.device):
        _check(lib.tdt_loss_fwd_bwd_ws(*args, _ptr(workspace), workspace.numel(),
                                       _stream_handle(logits.device)))
    return loss_out, grad_out


NOALLOC_MAX_WORKSPACE_BYTES = 64 * 1024 * 1024


def tdt_loss_fwd_bwd_noalloc(logits, labels, logit_lens, label_lens, durations, blank,
                             sigma=0.0, reduction="mean_volume", loss_out=None, grad_out=None,
                             compute_grad=True):
    """As tdt_loss_fwd_bwd, for callers that cannot allocate device memory.

    The library allocates nothing: its scratch is a fixed 64 MiB device array
    inside the library (problems needing more are rejected); every call on a
    device shares it, so order the calls on one stream.  Only the outputs
    are created here when not given -- pass loss_out and grad_out to
    allocate nothing at all.
    """
    args, loss_out, grad_out = _marshal(logits, labels, logit_lens, label_lens, durations,
                                        blank, sigma, reduction, loss_out, grad_out,
                                        compute_grad)
    with torch.cuda.device(logits.device):
        _check(lib.tdt_loss_fwd_bwd_noalloc(*args, _stream_handle(logits.device)))
    return loss_out, grad_out


# The calls of an attention decoder's steps are short: what follows keeps the host's part of them
# short too (packed argument arrays, the raw stream handle, no device switch where none is needed).
_NO_SWITCH = contextlib.nullcontext()
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else \
    torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_pack2, _pack3, _pack4, _pack6, _pack12, _pack24 = (
    struct.Struct("=%dq" % n).pack for n in (2, 3, 4, 6, 12, 24))


def _on(device):
    """The device's context, without the cost of a switch where it is current already."""
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device, not on %s" % device)
    return _NO_SWITCH if device.index == _current_device() else torch.cuda.device(device)


def tdt_cross_attn_workspace_size(sizes, dtype, backward: bool) -> int:
    """Bytes of scratch of a cross-attention call; sizes = (B, Lq, Lk, H, Hkv, D), dtype a torch
    dtype (0 for invalid arguments or when none is needed)."""
    return int(lib.tdt_cross_attn_workspace_size(_pack6(*sizes), DTYPES[dtype], int(backward)))


def _check_lens(name, t, B, dev):
    if t.dtype != torch.int64 or not t.is_contiguous() or t.device != dev or t.shape != (B,):
        raise ValueError("%s must be a contiguous int64 tensor of %d element(s) on %s"
                         % (name, B, dev))


def _attn_sizes(q, k, v, k_lens, q_lens, windows):
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("q must be [B, Lq, H, D], k and v [B, Lk, Hkv, D]")
    B, Lq, H, D = qs
    Bk, Lk, Hkv, Dk = ks
    if v.shape != ks or Bk != B or Dk != D:
        raise ValueError("k and v must be [B, Lk, Hkv, D] with q's B and D")
    dtype, dev = q.dtype, q.device
    if dtype not in DTYPES:
        raise TypeError("q dtype must be float32, float16 or bfloat16")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k and v must have one dtype")
    if k.device != dev or v.device != dev:
        raise ValueError("q, k and v must be on one device")
    if k_lens is not None:
        _check_lens("k_lens", k_lens, B, dev)
    if q_lens is not None:
        _check_lens("q_lens", q_lens, B, dev)
    if windows is not None and (windows.dtype != torch.int32 or not windows.is_contiguous()
                                or windows.device != dev or windows.shape != (B, Lq, 2)):
        raise ValueError("windows must be a contiguous int32 tensor [B, Lq, 2] on %s" % dev)
    return B, Lq, Lk, H, Hkv, D


def _rows(x):
    """(x, strides) with the elements of each head contiguous (a copy only where they are not)."""
    st = x.stride()
    if st[3] == 1 or x.shape[3] == 1:
        return x, st
    x = x.contiguous()
    return x, x.stride()


def _like(x, t, name):
    """(t, strides): checked to be an output of x's shape and dtype, or a new contiguous one."""
    if t is None:
        t = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        return t, t.stride()
    st = t.stride()
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device or (
            st[3] != 1 and t.shape[3] != 1):
        raise ValueError("%s must have the shape, dtype and device of its input and contiguous "
                         "heads" % name)
    return t, st


def _scratch(sizes, code, dev, backward, workspace):
    """(workspace, address, bytes): the given one, or a new one if the call needs any."""
    if workspace is None:
        need = lib.tdt_cross_attn_workspace_size(sizes, code, backward)
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif (workspace.dtype != torch.uint8 or workspace.device != dev
          or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    return workspace, workspace.data_ptr(), workspace.numel()


def tdt_cross_attn_fwd(q, k, v, k_lens=None, q_lens=None, windows=None, scale=None,
                       need_lse=True, out=None, lse=None, workspace=None):
    """Cross attention of label states q [B, Lq, H, D] to encoder frames k, v [B, Lk, Hkv, D] on
    the current CUDA stream (include/tdt_decoder.h, tdt_cross_attn_fwd); H a multiple of Hkv.

    k_lens, q_lens: int64 [B] or None (all); windows: int32 [B, Lq, 2], the frames [w0, w1) that
    each query sees, or None; scale: 1 / sqrt(D) unless given.  Few rows (decoding steps, the
    hypotheses of a beam) take the same call.  Any strides with contiguous heads, such as slices
    of a fused projection.  workspace: a contiguous uint8 tensor of
    tdt_cross_attn_workspace_size bytes at least, allocated unless given.  Returns (out, lse): out like q, lse float32 [B, H, Lq] (None without
    need_lse), which tdt_cross_attn_bwd takes.
    """
    B, Lq, Lk, H, Hkv, D = dims = _attn_sizes(q, k, v, k_lens, q_lens, windows)
    (q, sq), (k, sk), (v, sv) = _rows(q), _rows(k), _rows(v)
    out, so = _like(q, out, "out")
    dev = q.device
    if lse is not None:
        if (lse.dtype != torch.float32 or lse.shape != (B, H, Lq) or not lse.is_contiguous()
                or lse.device != dev):
            raise ValueError("lse must be a contiguous float32 tensor [B, H, Lq] on %s" % dev)
    elif need_lse:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=dev)
    sizes, code = _pack6(*dims), DTYPES[q.dtype]
    workspace, ws, nbytes = _scratch(sizes, code, dev, 0, workspace)
    with _on(dev):
        _check(lib.tdt_cross_attn_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), sizes,
            _pack12(*sq[:3], *sk[:3], *sv[:3], *so[:3]), code, _addr(k_lens), _addr(q_lens),
            _addr(windows), D ** -0.5 if scale is None else scale, out.data_ptr(), _addr(lse), ws,
            nbytes, _raw_stream(dev.index)))
    return out, lse


def tdt_cross_attn_bwd(grad_out, q, k, v, out, lse, k_lens=None, q_lens=None, windows=None,
                       scale=None, dq=None, dk=None, dv=None, workspace=None):
    """Gradients (dq, dk, dv) of sum(grad_out * out); out and lse are tdt_cross_attn_fwd's, the
    other arguments its own.  dq, dk, dv may be given, e.g. as slices of the gradient of a fused
    projection."""
    B, Lq, Lk, H, Hkv, D = dims = _attn_sizes(q, k, v, k_lens, q_lens, windows)
    dev = q.device
    for name, t in (("grad_out", grad_out), ("out", out)):
        if t.shape != q.shape or t.dtype != q.dtype or t.device != dev:
            raise ValueError("%s must have q's shape, dtype and device" % name)
    if (lse.dtype != torch.float32 or lse.shape != (B, H, Lq) or not lse.is_contiguous()
            or lse.device != dev):
        raise ValueError("lse must be a contiguous float32 tensor [B, H, Lq] on %s" % dev)
    (q, sq), (k, sk), (v, sv) = _rows(q), _rows(k), _rows(v)
    (out, so), (grad_out, sg) = _rows(out), _rows(grad_out)
    (dq, sdq), (dk, sdk), (dv, sdv) = _like(q, dq, "dq"), _like(k, dk, "dk"), _like(v, dv, "dv")
    sizes, code = _pack6(*dims), DTYPES[q.dtype]
    workspace, ws, nbytes = _scratch(sizes, code, dev, 1, workspace)
    with _on(dev):
        _check(lib.tdt_cross_attn_bwd(
            grad_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
            lse.data_ptr(), sizes,
            _pack24(*sq[:3], *sk[:3], *sv[:3], *so[:3], *sg[:3], *sdq[:3], *sdk[:3], *sdv[:3]),
            code, _addr(k_lens), _addr(q_lens), _addr(windows),
            D ** -0.5 if scale is None else scale, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws,
            nbytes, _raw_stream(dev.index)))
    return dq, dk, dv


def _setting(x, dtype, N, dev, name):
    """(device pointer or None, value) of a setting that is one number or a tensor [N]."""
    if not isinstance(x, torch.Tensor):
        return None, x
    if x.dtype != dtype or x.shape != (N,) or not x.is_contiguous() or x.device != dev:
        raise ValueError("%s must be a number or a contiguous %s tensor of %d element(s) on %s"
                         % (name, dtype, N, dev))
    return x.data_ptr(), None


def tdt_sample(logits, uniforms, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None,
               logprobs=None):
    """Draws a token of each row of ``logits`` [N, V] from ``uniforms`` (float32 [N], in [0, 1))
    on the current CUDA stream (include/tdt_decoder.h, tdt_sample): temperature (0: argmax),
    top_k (0: off), top_p (1: off), min_p (0: off), each a number or a tensor [N] (float32;
    top_k int32).  Rows may be a slice of wider ones, e.g. the token logits of joint outputs.
    Returns (tokens int32 [N], logprobs float32 [N]): the log-probability among the tokens that
    the filters leave."""
    if logits.dim() != 2:
        raise ValueError("logits must be [N, V]")
    if logits.dtype not in DTYPES:
        raise TypeError("logits dtype must be float32, float16 or bfloat16")
    N, V = logits.shape
    dev = logits.device
    if logits.stride(1) != 1 and V != 1:
        logits = logits.contiguous()
    if (uniforms.dtype != torch.float32 or uniforms.shape != (N,) or uniforms.device != dev
            or not uniforms.is_contiguous()):
        raise ValueError("uniforms must be a contiguous float32 tensor of %d element(s) on %s"
                         % (N, dev))
    f = torch.float32
    ts, t = _setting(temperature, f, N, dev, "temperature")
    ks, k = _setting(top_k, torch.int32, N, dev, "top_k")
    ps, p = _setting(top_p, f, N, dev, "top_p")
    ms, m = _setting(min_p, f, N, dev, "min_p")
    for name, x, dtype in (("tokens", tokens, torch.int32), ("logprobs", logprobs, f)):
        if x is not None and (x.dtype != dtype or x.shape != (N,) or not x.is_contiguous()
                              or x.device != dev):
            raise ValueError("%s must be a contiguous %s tensor of %d element(s) on %s"
                             % (name, dtype, N, dev))
    if tokens is None:
        tokens = torch.empty(N, dtype=torch.int32, device=dev)
    if logprobs is None:
        logprobs = torch.empty(N, dtype=f, device=dev)
    with _on(dev):
        _check(lib.tdt_sample(
            logits.data_ptr(), _pack2(N, V), logits.stride(0), DTYPES[logits.dtype],
            uniforms.data_ptr(), ts, ks, ps, ms, 1.0 if t is None else t, 0 if k is None else k,
            1.0 if p is None else p, 0.0 if m is None else m, tokens.data_ptr(),
            logprobs.data_ptr(), _raw_stream(dev.index)))
    return tokens, logprobs


# ---- the paged cache of label states --------------------------------------------------------------
E4M3 = torch.float8_e4m3fn
_CACHE_DTYPES = {**DTYPES, E4M3: 3}
_pack_cache = struct.Struct("=4Q4q12qi4x").pack  # tdt_paged_cache


class PagedCache:
    """Keys and values of label states in pages (include/tdt_decoder.h, tdt_paged_cache).

    k, v: [n_pages, page_size, heads, head_dim] of float32, float16, bfloat16 or float8_e4m3fn, any
    strides with contiguous rows (slices of one tensor, heads before places); page_size a power of
    two.  k_scales, v_scales: uint8 [n_pages, page_size, heads], with float8_e4m3fn only: a row
    stands for e4m3 * 2^(byte - 127).  ``PagedCache.empty`` allocates them.  Which pages an utterance
    has says its row of the page table that the calls take.
    """

    __slots__ = ("k", "v", "k_scales", "v_scales", "dtype", "device", "at", "page_size", "heads",
                 "head_dim", "_packed")

    def __init__(self, k, v, k_scales=None, v_scales=None):
        shape, dtype, dev = k.shape, k.dtype, k.device
        if len(shape) != 4 or v.shape != shape:
            raise ValueError("k and v must be [n_pages, page_size, heads, head_dim]")
        if dtype not in _CACHE_DTYPES:
            raise TypeError("pages must be float32, float16, bfloat16 or float8_e4m3fn")
        if v.dtype != dtype or v.device != dev:
            raise ValueError("k and v must have one dtype and device")
        sk, sv = k.stride(), v.stride()
        if (sk[3] != 1 or sv[3] != 1) and shape[3] != 1:
            raise ValueError("the elements of a row of pages must be contiguous")
        if dtype == E4M3:
            for t in (k_scales, v_scales):
                if t is None or t.dtype != torch.uint8 or t.shape != shape[:3] or t.device != dev:
                    raise ValueError("k_scales and v_scales must be uint8 [n_pages, page_size, heads] "
                                     "on %s" % dev)
            ks, vs = k_scales.data_ptr(), v_scales.data_ptr()
            strides = sk[:3] + sv[:3] + k_scales.stride() + v_scales.stride()
        elif k_scales is not None or v_scales is not None:
            raise ValueError("only pages of float8_e4m3fn have scales")
        else:
            ks = vs = 0
            strides = sk[:3] + sv[:3] + (0,) * 6
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.dtype, self.device, self.at = dtype, dev, k.get_device()
        self.page_size, self.heads, self.head_dim = shape[1:]
        self._packed = _pack_cache(k.data_ptr(), v.data_ptr(), ks, vs, *shape, *strides,
                                   _CACHE_DTYPES[dtype])

    @classmethod
    def empty(cls, n_pages, page_size, heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of new pages, whose contents are not set."""
        k, v = (torch.empty((n_pages, page_size, heads, head_dim), dtype=dtype, device=device)
                for _ in range(2))
        if dtype != E4M3:
            return cls(k, v)
        return cls(k, v, *(torch.empty((n_pages, page_size, heads), dtype=torch.uint8, device=device)
                           for _ in range(2)))


def _check_pages(cache, page_table, kv_lens, q_lens, B, dev):
    """(address, row stride, columns) of the page table."""
    if cache.device != dev:
        raise ValueError("the cache must be on %s" % dev)
    shape, stride = page_table.shape, page_table.stride()
    if (len(shape) != 2 or shape[0] != B or page_table.dtype != torch.int32
            or page_table.get_device() != cache.at or (stride[1] != 1 and shape[1] > 1)):
        raise ValueError("page_table must be an int32 tensor [%d, max_pages] with contiguous rows on %s"
                         % (B, dev))
    for name, t in (("kv_lens", kv_lens), ("q_lens", q_lens)):
        if t is not None and (t.dtype != torch.int64 or t.shape != (B,) or t.get_device() != cache.at
                              or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous int64 tensor of %d element(s) on %s"
                             % (name, B, dev))
    return page_table.data_ptr(), stride[0], shape[1]


def _out_rows(t, shape, dtype, dev, name):
    """(t, strides): checked to be an output with contiguous rows, or a new contiguous one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
    elif t.shape != shape or t.dtype != dtype or t.device != dev or (t.stride(-1) != 1 and shape[-1] != 1):
        raise ValueError("%s must be %s of %s on %s with contiguous rows" % (name, tuple(shape), dtype, dev))
    return t, t.stride()


def tdt_cache_write(k, v, cache, page_table, kv_lens, q_lens=None):
    """Writes new label states' k, v [B, L, heads, head_dim] into the pages of ``cache`` on the current
    CUDA stream (include/tdt_decoder.h, tdt_cache_write); float8_e4m3fn pages are quantised as they
    are written.

    Row i < q_lens[b] of utterance b is position kv_lens[b] - q_lens[b] + i: kv_lens (int64 [B]) counts
    the new rows; q_lens: int64 [B] or None (all L).  page_table: int32 [B, max_pages].  k and v may
    be slices of a fused projection.
    """
    ks, dtype, dev = k.shape, k.dtype, cache.device
    if len(ks) != 4 or v.shape != ks or ks[2] != cache.heads or ks[3] != cache.head_dim:
        raise ValueError("k and v must be [B, L, %d, %d]" % (cache.heads, cache.head_dim))
    if dtype not in DTYPES or v.dtype != dtype:
        raise TypeError("k and v must be float32, float16 or bfloat16, of one dtype")
    if cache.dtype != dtype and cache.dtype != E4M3:
        raise TypeError("pages of %s cannot hold rows of %s" % (cache.dtype, dtype))
    if k.get_device() != cache.at or v.get_device() != cache.at:
        raise ValueError("k, v and the cache must be on one device")
    table, stride, columns = _check_pages(cache, page_table, kv_lens, q_lens, ks[0], dev)
    (k, sk), (v, sv) = _rows(k), _rows(v)
    with _on(dev):
        _check(lib.tdt_cache_write(
            k.data_ptr(), v.data_ptr(), _pack3(ks[0], ks[1], columns), _pack6(*sk[:3], *sv[:3]),
            DTYPES[dtype], cache._packed, table, stride, kv_lens.data_ptr(), _addr(q_lens),
            _raw_stream(dev.index)))


def tdt_cache_read(cache, page_table, kv_lens, q_lens, length, dtype, k=None, v=None):
    """Rows of ``cache`` as (k, v), each [B, length, heads, head_dim] of ``dtype``: row i < q_lens[b] of
    utterance b is position kv_lens[b] - q_lens[b] + i, as in tdt_cache_write (q_lens = kv_lens: whole
    utterances; None: all ``length``); later rows are 0.  k and v may be given."""
    B, dev = kv_lens.shape[0], cache.device
    if dtype not in DTYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    table, stride, columns = _check_pages(cache, page_table, kv_lens, q_lens, B, dev)
    shape = (B, length, cache.heads, cache.head_dim)
    k, sk = _out_rows(k, shape, dtype, dev, "k")
    v, sv = _out_rows(v, shape, dtype, dev, "v")
    with _on(dev):
        _check(lib.tdt_cache_read(
            cache._packed, table, stride, kv_lens.data_ptr(), _addr(q_lens), _pack3(B, length, columns),
            _pack6(*sk[:3], *sv[:3]), DTYPES[dtype], k.data_ptr(), v.data_ptr(), _raw_stream(dev.index)))
    return k, v


def tdt_paged_attn_workspace_size(sizes, dtype, cache) -> int:
    """Bytes of scratch of tdt_paged_attn; sizes = (B, Lq, H, max_pages), dtype q's (0 for invalid
    arguments or when none is needed)."""
    return int(lib.tdt_paged_attn_workspace_size(_pack4(*sizes), DTYPES[dtype], cache._packed))


def tdt_paged_attn(q, cache, page_table, kv_lens, q_lens=None, scale=None, need_lse=False, out=None,
                   lse=None, workspace=None):
    """Causal attention of new label states q [B, Lq, H, D] over the pages of ``cache``, which hold their
    own keys and values already (tdt_cache_write of the same lengths), on the current CUDA stream
    (include/tdt_decoder.h, tdt_paged_attn); H a multiple of the cache's heads.

    Query i < q_lens[b] of utterance b is at position kv_lens[b] - q_lens[b] + i and sees the positions
    up to its own; queries past q_lens[b] (None: all Lq) get 0.  Pages are of q's dtype or
    float8_e4m3fn.  scale: 1 / sqrt(D) unless given.  workspace: a contiguous uint8 tensor of
    tdt_paged_attn_workspace_size bytes at least, allocated unless given; where calls need one it may go
    with the page table's width, so pass a table no wider than needed.  Returns (out, lse): out like q,
    lse float32 [B, H, Lq], or None without need_lse.
    """
    shape, dtype, dev = q.shape, q.dtype, cache.device
    if len(shape) != 4 or shape[3] != cache.head_dim:
        raise ValueError("q must be [B, Lq, H, %d]" % cache.head_dim)
    if dtype not in DTYPES:
        raise TypeError("q dtype must be float32, float16 or bfloat16")
    if cache.dtype != dtype and cache.dtype != E4M3:
        raise TypeError("queries of %s cannot read pages of %s" % (dtype, cache.dtype))
    if q.get_device() != cache.at:
        raise ValueError("q and the cache must be on one device")
    B, Lq, H, D = shape
    table, stride, columns = _check_pages(cache, page_table, kv_lens, q_lens, B, dev)
    q, sq = _rows(q)
    out, so = _out_rows(out, shape, dtype, dev, "out")
    if lse is not None:
        if (lse.dtype != torch.float32 or lse.shape != (B, H, Lq) or not lse.is_contiguous()
                or lse.device != dev):
            raise ValueError("lse must be a contiguous float32 tensor [B, H, Lq] on %s" % dev)
    elif need_lse:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=dev)
    sizes, code, ws, nbytes = _pack4(B, Lq, H, columns), DTYPES[dtype], None, 0
    if workspace is None:
        nbytes = lib.tdt_paged_attn_workspace_size(sizes, code, cache._packed)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            ws = workspace.data_ptr()
    elif (workspace.dtype != torch.uint8 or workspace.device != dev
          or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    else:
        ws, nbytes = workspace.data_ptr(), workspace.numel()
    with _on(dev):
        _check(lib.tdt_paged_attn(
            q.data_ptr(), sizes, _pack6(*sq[:3], *so[:3]), code, cache._packed, table, stride,
            kv_lens.data_ptr(), _addr(q_lens), D ** -0.5 if scale is None else scale, out.data_ptr(),
            _addr(lse), ws, nbytes, _raw_stream(dev.index)))
    return out, lse


# ---- log-probabilities of given tokens --------------------------------------------------------------
class TokenLogprobs(NamedTuple):
    """logprobs, entropy float32 [N]; stats float32 [N, 2]: each row's maximum m and
    ln sum exp(x - m); top_tokens int32, top_logprobs float32 [N, n_top] (None without)."""

    logprobs: torch.Tensor
    entropy: torch.Tensor
    stats: torch.Tensor
    top_tokens: Optional[torch.Tensor] = None
    top_logprobs: Optional[torch.Tensor] = None


def _check_scored(logits, tokens):
    """(logits with contiguous rows, N, V, row stride)"""
    shape, stride = logits.shape, logits.stride()
    if len(shape) != 2:
        raise ValueError("logits must be [N, V]")
    if logits.dtype not in DTYPES:
        raise TypeError("logits dtype must be float32, float16 or bfloat16")
    N, V = shape
    if (tokens.dtype != torch.int64 or tokens.shape != (N,) or not tokens.is_contiguous()
            or tokens.get_device() != logits.get_device()):
        raise ValueError("tokens must be a contiguous int64 tensor of %d element(s) on %s"
                         % (N, logits.device))
    if stride[1] != 1 and V != 1:
        logits = logits.contiguous()
        stride = logits.stride()
    return logits, N, V, stride[0]


def _new_logprobs(N, n_top, dev):
    f = torch.float32
    three = (torch.empty(N, dtype=f, device=dev), torch.empty(N, dtype=f, device=dev),
             torch.empty((N, 2), dtype=f, device=dev))
    if not n_top:
        return TokenLogprobs(*three)
    n_top = max(0, n_top)  # a negative one is refused with the other arguments
    return TokenLogprobs(*three, torch.empty((N, n_top), dtype=torch.int32, device=dev),
                         torch.empty((N, n_top), dtype=f, device=dev))


def _weights(t, N, at, name):
    """Address of weights (None: none); at: the logits' device index."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != (N,) or t.get_device() != at or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of %d element(s) on the logits' device"
                         % (name, N))
    return t.data_ptr()


def _grad_rows(logits, grad_out):
    if grad_out is None:
        return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    if (grad_out.shape != logits.shape or grad_out.dtype != logits.dtype
            or grad_out.device != logits.device or (grad_out.stride(1) != 1 and logits.shape[1] != 1)):
        raise ValueError("grad_out must have the logits' shape, dtype and device and contiguous rows")
    return grad_out


def tdt_token_logprobs_fwd(logits, tokens, n_top=0):
    """Log-probability of ``tokens`` (int64 [N]; negative: padding, the row takes no part) under each row
    of ``logits`` [N, V], the row's entropy, and its ``n_top`` most probable tokens, on the current
    CUDA stream (include/tdt_decoder.h, tdt_token_logprobs_fwd).  Rows may be a slice of wider ones.
    Returns TokenLogprobs."""
    logits, N, V, stride = _check_scored(logits, tokens)
    dev = logits.device
    r = _new_logprobs(N, n_top, dev)
    with _on(dev):
        _check(lib.tdt_token_logprobs_fwd(
            logits.data_ptr(), _pack3(N, V, n_top), stride, DTYPES[logits.dtype],
            tokens.data_ptr(), r.logprobs.data_ptr(), r.entropy.data_ptr(), r.stats.data_ptr(),
            _addr(r.top_tokens), _addr(r.top_logprobs), _raw_stream(dev.index)))
    return r


def tdt_token_logprobs_bwd(logits, tokens, result, grad_logprobs=None, grad_entropy=None, grad_top=None,
                           grad_out=None):
    """The logits' gradient, [N, V] of their dtype, for weights grad_logprobs, grad_entropy (float32 [N])
    and grad_top (float32 [N, n_top]) of ``result``, which tdt_token_logprobs_fwd returned for the same
    logits and tokens.  grad_out may be ``logits``: the gradient then replaces them."""
    rows = logits
    logits, N, V, stride = _check_scored(logits, tokens)
    dev = logits.device
    at = logits.get_device()
    a, b = _weights(grad_logprobs, N, at, "grad_logprobs"), _weights(grad_entropy, N, at, "grad_entropy")
    entropy = _weights(result.entropy, N, at, "entropy")
    stats, top, n_top = result.stats, result.top_tokens, 0
    if (stats.dtype != torch.float32 or stats.shape != (N, 2) or not stats.is_contiguous()
            or stats.device != dev):
        raise ValueError("stats must be a contiguous float32 tensor [%d, 2] on %s" % (N, dev))
    if grad_top is not None:
        if top is None:
            raise ValueError("grad_top is of alternatives that the result does not hold")
        for name, t, dtype in (("grad_top", grad_top, torch.float32), ("top_tokens", top, torch.int32)):
            if (t.dtype != dtype or t.shape != top.shape or t.dim() != 2 or t.shape[0] != N
                    or not t.is_contiguous() or t.device != dev):
                raise ValueError("%s must be a contiguous %s tensor [%d, n_top] on %s"
                                 % (name, dtype, N, dev))
        n_top = top.shape[1]
    grad_out = _grad_rows(rows, grad_out)
    with _on(dev):
        _check(lib.tdt_token_logprobs_bwd(
            logits.data_ptr(), _pack3(N, V, n_top), _pack2(stride, grad_out.stride(0)),
            DTYPES[logits.dtype], tokens.data_ptr(), entropy, stats.data_ptr(), _addr(top), a, b,
            _addr(grad_top), grad_out.data_ptr(), _raw_stream(dev.index)))
    return grad_out


def tdt_token_logprobs_fwd_bwd(logits, tokens, grad_logprobs=None, grad_entropy=None, n_top=0,
                               grad_out=None):
    """Both in one call, for weights that are known beforehand: (TokenLogprobs, gradient of the logits).
    Arguments as of tdt_token_logprobs_fwd and tdt_token_logprobs_bwd."""
    rows = logits
    logits, N, V, stride = _check_scored(logits, tokens)
    dev = logits.device
    at = logits.get_device()
    a, b = _weights(grad_logprobs, N, at, "grad_logprobs"), _weights(grad_entropy, N, at, "grad_entropy")
    grad_out = _grad_rows(rows, grad_out)
    r = _new_logprobs(N, n_top, dev)
    with _on(dev):
        _check(lib.tdt_token_logprobs_fwd_bwd(
            logits.data_ptr(), _pack3(N, V, n_top), _pack2(stride, grad_out.stride(0)),
            DTYPES[logits.dtype], tokens.data_ptr(), a, b, r.logprobs.data_ptr(), r.entropy.data_ptr(),
            r.stats.data_ptr(), _addr(r.top_tokens), _addr(r.top_logprobs), grad_out.data_ptr(),
            _raw_stream(dev.index)))
    return r, grad_out


def _new_workspace(logits, n_dur):
    return torch.empty(max(1, workspace_size(logits.shape, n_dur)), dtype=torch.uint8,
                       device=logits.device)


def tdt_loss_fwd(logits, labels, logit_lens, label_lens, durations, blank, sigma=0.0,
                 reduction="mean_volume", loss_out=None, workspace=None):
    """Forward half of the split API: returns (loss, workspace).

    The workspace (a uint8 CUDA tensor, created when not given) holds what
    tdt_loss_bwd needs; keep it untouched until then.
    """
    args, loss_out, _ = _marshal(logits, labels, logit_lens, label_lens, durations, blank, sigma,
                                 reduction, loss_out, None, False)
    if workspace is None:
        workspace = _new_workspace(logits, len(durations))
    _check_workspace(workspace, logits.device)
    with torch.cuda.device(logits.device):
        _check(lib.tdt_loss_fwd(*args[:-1], _ptr(workspace), workspace.numel(),
                                _stream_handle(logits.device)))
    return loss_out, workspace


def tdt_loss_bwd(logits, labels, logit_lens, label_lens, durations, blank, workspace,
                 grad_loss=None, sigma=0.0, reduction="mean_volume", grad_out=None):
    """Backward half: the gradient for upstream gradient ``grad_loss``.

    ``grad_loss``: float32 CUDA tensor with B elements ("none") or one
    element, or None for 1.  Arguments other than grad_loss/grad_out must be
    those of the tdt_loss_fwd call that filled ``workspace``.  ``grad_out``
    may be ``logits`` itself (contiguous logits): the gradient then replaces
    them.
    """
    _check_workspace(workspace, logits.device)
    B = logits.shape[0]
    if grad_loss is not None:
        want = B if reduction == "none" else 1
        if (grad_loss.dtype != torch.float32 or not grad_loss.is_contiguous()
                or grad_loss.numel() != want or grad_loss.device != logits.device):
            raise ValueError("grad_loss must be a contiguous float32 tensor of %d element(s) "
                             "on %s" % (want, logits.device))
    args, _, grad_out = _marshal(logits, labels, logit_lens, label_lens, durations, blank, sigma,
                                 reduction, None, grad_out, True, with_loss=False)
    with torch.cuda.device(logits.device):
        _check(lib.tdt_loss_bwd(*args[:-2], _ptr(grad_loss), args[-1], _ptr(workspace),
                                workspace.numel(), _stream_handle(logits.device)))
    return grad_out


def tdt_loss_workspace_size(sizes, n_dur: int) -> int:
    """Bytes of scratch tdt_loss_fwd_bwd_ws needs (0 for invalid sizes)."""
    return workspace_size(sizes, n_dur)


def tdt_status_string(status: int) -> str:
    return status_string(status)


def tdt_loss_version() -> int:
    return int(lib.tdt_loss_version())


def tdt_loss_set_lattice_bands(bands: int) -> int:
    """Force K bands (CTAs per utterance and direction) in the lattice passes;
    0 = automatic.  Results do not depend on K.  Returns the previous value."""
    return int(lib.tdt_loss_set_lattice_bands(int(bands)))


def tdt_loss_set_lattice_exchange(mode: int) -> int:
    """How lattice bands exchange boundary rows: 0 = automatic, 1 = a
    thread-block cluster, 2 = global memory.  Results do not depend on it.
    Returns the previous value."""
    return int(lib.tdt_loss_set_lattice_exchange(int(mode)))


def tdt_loss_test_set_halo_fault(utterance: int, wait_limit_cycles: int = 0) -> int:
    """Testing: make the multi-band lattice passes of utterance index
    ``utterance`` lose their band-1 boundary row so the neighbours' bounded
    waits run out (NaN loss, zero gradient rows for that utterance only);
    ``wait_limit_cycles`` > 0 shortens every wait's limit.  utterance < 0
    switches it off.  Returns the previous utterance setting."""
    return int(lib.tdt_loss_test_set_halo_fault(int(utterance), int(wait_limit_cycles)))


KERNEL_NAMES = ("node_tables", "lattice", "reduce", "grad")


def tdt_loss_timing_enable(on: bool) -> None:
    """Record CUDA events around each kernel of later calls (benchmarks only)."""
    lib.tdt_loss_timing_enable(1 if on else 0)


def tdt_loss_timing_read(reset: bool = True):
    """{kernel name: (summed ms, launches, summed busy-window ms)} since the
    last reset; waits for the events.  The busy window of a kernel in one call
    runs from the start of its first launch to the end of its last (launches
    on several streams may overlap)."""
    n = len(KERNEL_NAMES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    span = (ctypes.c_double * n)()
    rc = lib.tdt_loss_timing_read(ms, cnt, span, n, 1 if reset else 0)
    if rc < 0:
        raise TDTError(rc, status_string(rc))
    return {KERNEL_NAMES[i]: (ms[i], cnt[i], span[i]) for i in range(n)}
