"""Cross attention and sampling refuse bad arguments on the host, before touching any device
(no GPU here: only calls that fail validation, or have nothing to do, are made)."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from transducer_loss_asr_gb300 import build

    build.build()
    from transducer_loss_asr_gb300 import binding

    return binding


def _strides(B, L, H, D):
    return [L * H * D, H * D, D]


def _attn(lib, backward, **over):
    a = dict(sizes=[2, 5, 7, 4, 2, 64], dtype=2, scale=0.125, q=FAKE, k=FAKE, v=FAKE, out=FAKE,
             lse=FAKE, k_lens=FAKE, q_lens=FAKE, windows=FAKE, go=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             workspace=None, workspace_bytes=None, strides=None)
    a.update(over)
    sizes = None if a["sizes"] is None else (ctypes.c_int64 * 6)(*a["sizes"])
    n = 8 if backward else 4
    if a["strides"] is None:
        B, Lq, Lk, H, Hkv, D = a["sizes"] or [2, 5, 7, 4, 2, 64]
        qs, ks = _strides(B, Lq, H, D), _strides(B, Lk, Hkv, D)
        flat = (qs + ks + ks + qs + qs + qs + ks + ks)[: 3 * n]
        for at, value in a.get("stride_at", {}).items():
            flat[at] = value
        strides = (ctypes.c_int64 * (3 * n))(*flat)
    else:
        strides = None
    need = 0 if sizes is None else lib.lib.tdt_cross_attn_workspace_size(sizes, a["dtype"],
                                                                         int(backward))
    nb = need if a["workspace_bytes"] is None else a["workspace_bytes"]
    ws = FAKE if a["workspace"] is None else a["workspace"]
    if backward:
        return lib.lib.tdt_cross_attn_bwd(a["go"], a["q"], a["k"], a["v"], a["out"], a["lse"], sizes,
                                          strides, a["dtype"], a["k_lens"], a["q_lens"],
                                          a["windows"], a["scale"], a["dq"], a["dk"], a["dv"], ws,
                                          nb, None)
    return lib.lib.tdt_cross_attn_fwd(a["q"], a["k"], a["v"], sizes, strides, a["dtype"],
                                      a["k_lens"], a["q_lens"], a["windows"], a["scale"], a["out"],
                                      a["lse"], ws, nb, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(sizes=None), -1),
    (dict(strides="none"), -1),
    (dict(q=None), -1),
    (dict(k=None), -1),
    (dict(v=None), -1),
    (dict(out=None), -1),
    (dict(sizes=[-1, 5, 7, 4, 2, 64]), -2),
    (dict(sizes=[2, -5, 7, 4, 2, 64]), -2),
    (dict(sizes=[2, 5, 1 << 30, 4, 2, 64]), -2),
    (dict(sizes=[1 << 20, 5, 1 << 20, 4, 2, 64]), -2),
    (dict(stride_at={0: -1}), -3),
    (dict(dtype=3), -4),
    (dict(q=FAKE + 1), -11),
    (dict(k=FAKE + 1), -11),
    (dict(lse=FAKE + 2), -11),
    (dict(windows=FAKE + 4), -11),
    (dict(k_lens=FAKE + 4), -11),
    (dict(sizes=[2, 5, 7, 4, 3, 64]), -14),   # H not a multiple of Hkv
    (dict(sizes=[2, 5, 7, 0, 0, 64]), -14),
    (dict(sizes=[2, 5, 7, 4, 2, 0]), -14),
    (dict(sizes=[2, 5, 7, 4, 2, 257]), -14),
    (dict(scale=0.0), -15),
    (dict(scale=-0.5), -15),
    (dict(scale=float("nan")), -15),
    (dict(scale=float("inf")), -15),
])
def test_cross_attention_refuses(lib, backward, over, code):
    assert _attn(lib, backward, **over) == code


def test_cross_attention_refuses_outputs_that_overlap_themselves(lib):
    assert _attn(lib, False, stride_at={11: 32}) == -3         # heads of out overlap
    assert _attn(lib, False, stride_at={9: 64}) == -3
    for at in (17, 20, 23):                                    # dq, dk, dv
        assert _attn(lib, True, stride_at={at: 0}) == -3


def test_cross_attention_backward_refuses_missing_pieces(lib):
    for name in ("go", "lse", "dq", "dk", "dv"):
        assert _attn(lib, True, **{name: None}) == -1
    need = lib.tdt_cross_attn_workspace_size([2, 5, 7, 4, 2, 64], torch.bfloat16, True)
    assert need > 0
    assert _attn(lib, True, workspace_bytes=need - 1) == -9
    assert _attn(lib, True, workspace=FAKE + 8) == -11
    assert _attn(lib, True, workspace=0) == -1


def test_cross_attention_with_nothing_to_do(lib):
    assert _attn(lib, False, sizes=[0, 5, 7, 4, 2, 64]) == 0
    assert _attn(lib, False, sizes=[2, 0, 7, 4, 2, 64]) == 0
    assert _attn(lib, True, sizes=[0, 5, 7, 4, 2, 64]) == 0
    assert _attn(lib, True, sizes=[2, 0, 0, 4, 2, 64]) == 0
    assert lib.tdt_cross_attn_workspace_size([2, 5, 7, 4, 3, 64], torch.bfloat16, True) == 0


def test_binding_refuses_bad_attention_tensors(lib):
    q, k = torch.zeros(2, 5, 4, 8), torch.zeros(2, 7, 2, 8)
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(q[0], k, k)
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(q, k, k[:, :6])
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(q, k[..., :4], k[..., :4])
    with pytest.raises(TypeError):
        lib.tdt_cross_attn_fwd(q.double(), k.double(), k.double())
    with pytest.raises(TypeError):
        lib.tdt_cross_attn_fwd(q, k.half(), k)
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(q, k, k, k_lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(q, k, k, q_lens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(q, k, k, windows=torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(q, k, k, out=torch.zeros(2, 5, 4, 4))
    lse = torch.zeros(2, 4, 5)
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_bwd(q[:, :4], q, k, k, q, lse)
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_bwd(q, q, k, k, q, lse.double())


def _sample(lib, **over):
    a = dict(logits=FAKE, sizes=[3, 50], stride=50, dtype=0, u=FAKE, ts=None, ks=None, ps=None,
             ms=None, t=1.0, k=0, p=1.0, m=0.0, tokens=FAKE, logprobs=FAKE)
    a.update(over)
    sizes = None if a["sizes"] is None else (ctypes.c_int64 * 2)(*a["sizes"])
    return lib.lib.tdt_sample(a["logits"], sizes, a["stride"], a["dtype"], a["u"], a["ts"], a["ks"],
                              a["ps"], a["ms"], a["t"], a["k"], a["p"], a["m"], a["tokens"],
                              a["logprobs"], None)


@pytest.mark.parametrize("over,code", [
    (dict(sizes=None), -1),
    (dict(logits=None), -1),
    (dict(u=None), -1),
    (dict(tokens=None), -1),
    (dict(sizes=[-1, 50]), -2),
    (dict(sizes=[3, 0]), -2),
    (dict(sizes=[3, (1 << 24) + 1]), -2),
    (dict(stride=-50), -3),
    (dict(dtype=3), -4),
    (dict(logits=FAKE + 2), -11),
    (dict(logits=FAKE + 1, dtype=2), -11),
    (dict(u=FAKE + 2), -11),
    (dict(ts=FAKE + 2), -11),
    (dict(t=-0.1), -16),
    (dict(t=float("nan")), -16),
    (dict(t=float("inf")), -16),
    (dict(k=-1), -16),
    (dict(p=1.5), -16),
    (dict(p=-0.1), -16),
    (dict(m=2.0), -16),
    (dict(m=float("nan")), -16),
    (dict(sizes=[0, 50]), 0),
])
def test_sampling_refuses(lib, over, code):
    assert _sample(lib, **over) == code


def test_binding_refuses_bad_sampling_tensors(lib):
    x, u = torch.zeros(3, 50), torch.zeros(3)
    with pytest.raises(ValueError):
        lib.tdt_sample(x[0], u)
    with pytest.raises(TypeError):
        lib.tdt_sample(x.double(), u)
    with pytest.raises(ValueError):
        lib.tdt_sample(x, u[:2])
    with pytest.raises(ValueError):
        lib.tdt_sample(x, u, top_k=torch.zeros(3))            # int32 wanted
    with pytest.raises(ValueError):
        lib.tdt_sample(x, u, temperature=torch.zeros(2))
    with pytest.raises(ValueError):
        lib.tdt_sample(x, u, tokens=torch.zeros(3, dtype=torch.int64))


def test_new_status_texts(lib):
    for code in (-14, -15, -16):
        assert lib.tdt_status_string(code) != "unknown status"


def test_cross_attention_op_fake_shapes_and_cpu_rejection(lib):
    from transducer_loss_asr_gb300 import autograd

    q, k = torch.empty(2, 5, 4, 8, device="meta"), torch.empty(2, 7, 2, 8, device="meta")
    out, lse = torch.ops.tdt_gb300.cross_attention_forward(q, k, k, None, None, None, 0.3)
    assert out.shape == q.shape and lse.shape == (2, 4, 5) and lse.dtype == torch.float32
    grads = torch.ops.tdt_gb300.cross_attention_backward(q, q, k, k, out, lse, None, None, None, 0.3)
    assert [g.shape for g in grads] == [q.shape, k.shape, k.shape]
    with pytest.raises(NotImplementedError):  # CUDA kernels only: no silent CPU path
        autograd.cross_attention(torch.zeros(2, 5, 4, 8), torch.zeros(2, 7, 2, 8), torch.zeros(2, 7, 2, 8))
    with pytest.raises(ValueError):
        lib.tdt_cross_attn_fwd(torch.zeros(2, 5, 4, 8), torch.zeros(2, 7, 2, 8), torch.zeros(2, 7, 2, 8))


@pytest.mark.parametrize("workspace", [torch.zeros(1 << 20, dtype=torch.float32), torch.empty(1 << 20, dtype=torch.uint8, device="meta"),
                                       torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2]],
                         ids=["dtype", "device", "one byte", "strided"])
def test_binding_refuses_scratch_that_is_not_the_devices_own(lib, workspace):
    q, k = torch.zeros(2, 5, 4, 8), torch.zeros(2, 7, 2, 8)
    with pytest.raises(ValueError, match="workspace"):
        lib.tdt_cross_attn_fwd(q, k, k, workspace=workspace)
    with pytest.raises(ValueError, match="workspace"):
        lib.tdt_cross_attn_bwd(q, q, k, k, q, torch.zeros(2, 4, 5), workspace=workspace)
