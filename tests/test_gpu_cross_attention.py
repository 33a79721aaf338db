"""Cross attention on the GPU against the formulas in 64 bits.

Tolerances are bounds on what the kernels may round, worked out with the reference (see _reference): products and sums in float32 (unit 2^-24),
exponentials good to 2^-20, and for the 16-bit types one rounding each of the probabilities, of ds and of every result (unit u).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-30, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-30}  # least steps of the type
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transducer_loss_asr_gb300 import binding as b

    return b


def _reference(q, k, v, go, seen, scale, dtype):
    """{name: (value, bound)} in 64 bits; seen: truth values [B, Lq, Lk]."""
    B, Lq, H, D = q.shape
    G = H // k.shape[2]
    e32, u = 2.0 ** -24, UNIT[dtype]
    m = seen[:, None]
    rows, cols = seen.any(2), seen.any(1)
    q = torch.where(rows[:, :, None, None], q.double(), 0.0).transpose(1, 2)
    go = torch.where(rows[:, :, None, None], go.double(), 0.0).transpose(1, 2)
    k = torch.where(cols[:, :, None, None], k.double(), 0.0).transpose(1, 2).repeat_interleave(G, 1)
    v = torch.where(cols[:, :, None, None], v.double(), 0.0).transpose(1, 2).repeat_interleave(G, 1)
    Lk = k.shape[2]
    s = torch.where(m, q @ k.transpose(2, 3) * scale, -math.inf)
    lse = torch.logsumexp(s, 3) if Lk else torch.full((B, H, Lq), -math.inf, device=q.device).double()
    p = torch.where(m, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    out = p @ v
    # relative error of a probability: of its score and of lse (D + 8 roundings of terms up to |q||k|), and the exponentials
    size = torch.where(m, q.abs() @ k.abs().transpose(2, 3) * scale, 0.0)
    most = size.amax(3) if Lk else torch.zeros_like(lse)
    ep = 2 * (D + 8 + Lk ** 0.5) * e32 * (most + 1.0) + 2.0 ** -20
    up = u if dtype != torch.float32 else 0.0
    pe = p * (ep[..., None] + up)
    tol_out = pe @ v.abs() + u * out.abs()
    dp = go @ v.transpose(2, 3)
    delta = (go * out).sum(3)
    ds = p * (dp - delta[..., None])
    e_dp = (D + 8) * e32 * (go.abs() @ v.abs().transpose(2, 3))
    e_delta = (go.abs() * tol_out).sum(3) + (D + 8) * e32 * (go.abs() * out.abs()).sum(3)
    dse = p * ep[..., None] * (dp - delta[..., None]).abs() + p * (e_dp + e_delta[..., None]) + up * ds.abs()
    acc = (Lk + Lq * G + 8) ** 0.5 * 4 * e32  # sums of that many terms, in whichever order

    def grouped(x):
        return x.reshape(B, H // G, G, Lk, D).sum(2)

    dq, dk, dv = scale * (ds @ k), grouped(scale * (ds.transpose(2, 3) @ q)), grouped(p.transpose(2, 3) @ go)
    t_dq = scale * ((dse + acc * ds.abs()) @ k.abs()) + u * dq.abs()
    t_dk = grouped(scale * ((dse + acc * ds.abs()).transpose(2, 3) @ q.abs())) + u * dk.abs()
    t_dv = grouped((pe + acc * p).transpose(2, 3) @ go.abs()) + u * dv.abs()
    tol_out = tol_out + acc * (p @ v.abs())
    t_lse = 2 * (D + 8) * e32 * (most + 1.0) + 2.0 ** -20 + 4 * e32 * torch.where(lse.isinf(), 0.0, lse.abs())
    r = dict(out=(out, tol_out), dq=(dq, t_dq), dk=(dk, t_dk), dv=(dv, t_dv))
    r = {n: (x.transpose(1, 2), t.transpose(1, 2) + 2 * TINY[dtype]) for n, (x, t) in r.items()}
    r["lse"] = (lse, t_lse)
    return r


def _seen(B, Lq, Lk, k_lens, q_lens, windows, dev):
    j = torch.arange(Lk, device=dev)
    m = torch.ones(B, Lq, Lk, dtype=torch.bool, device=dev)
    if k_lens is not None:
        m &= (j < k_lens[:, None])[:, None]
    if q_lens is not None:
        m &= (torch.arange(Lq, device=dev) < q_lens[:, None])[..., None]
    if windows is not None:
        m &= (j >= windows[..., :1]) & (j < windows[..., 1:])
    return m


def _inputs(shape, dtype, seed, lens=False, windows=False, fused=True, poison=True, std=1.0):
    B, Lq, Lk, H, Hkv, D = shape
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return (torch.randn(s, generator=g, device="cuda") * std).to(dtype)

    q, go = randn(B, Lq, H, D), randn(B, Lq, H, D)
    if fused:
        kv = randn(B, Lk, 2, Hkv, D)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = randn(B, Lk, Hkv, D), randn(B, Hkv, Lk, D).transpose(1, 2)
    a = dict(k_lens=None, q_lens=None, windows=None)
    if lens:
        a["k_lens"] = torch.randint(0, Lk + 1, (B,), generator=g, device="cuda")
        a["q_lens"] = torch.randint(0, Lq + 1, (B,), generator=g, device="cuda")
        a["k_lens"][0], a["q_lens"][0] = max(1, Lk - 3), max(1, Lq - 1)
        if B > 1:
            a["k_lens"][1] = 0
        if poison:  # what lies past the lengths may be anything
            for b in range(B):
                k[b, a["k_lens"][b]:], v[b, a["k_lens"][b]:] = math.nan, math.nan
                q[b, a["q_lens"][b]:], go[b, a["q_lens"][b]:] = math.nan, math.inf
    if windows:
        at = torch.randint(-20, Lk + 20, (B, Lq), generator=g, device="cuda", dtype=torch.int32)
        n = torch.randint(-3, 60, (B, Lq), generator=g, device="cuda", dtype=torch.int32)
        a["windows"] = torch.stack([at, at + n], -1).contiguous()
    return q, k, v, go, a


def _near(name, x, value, bound, record=None, case=""):
    x = x.double()
    assert torch.equal(x.isinf(), value.isinf()) and torch.equal(x.isnan(), value.isnan()), name
    fine = value.isfinite()
    if not fine.any():
        return
    ratio = ((x - value).abs()[fine] / bound[fine].clamp_min(1e-300)).max().item()
    if record:
        record(case, name, ratio, 1.0)
    assert ratio <= 1.0, "%s: error is %.3g of its bound" % (name, ratio)


def _check(binding, shape, dtype, seed=0, scale=None, record=None, case="", **how):
    B, Lq, Lk, H, Hkv, D = shape
    q, k, v, go, a = _inputs(shape, dtype, seed, **how)
    f = D ** -0.5 if scale is None else scale
    want = _reference(q, k, v, go, _seen(B, Lq, Lk, **a, dev=q.device), f, dtype)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, scale=scale, **a)
    dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, scale=scale, **a)
    got = dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)
    for name, (value, bound) in want.items():
        _near(name, got[name], value, bound, record, case)
    alone, none = binding.tdt_cross_attn_fwd(q, k, v, scale=scale, need_lse=False, **a)
    assert none is None and torch.equal(alone.nan_to_num(7.0), out.nan_to_num(7.0))


SHAPES = [
    (1, 1, 1, 1, 1, 8),          # one query, one frame
    (2, 1, 200, 8, 8, 64),       # a decoding step
    (3, 1, 333, 8, 2, 128),      # a step of shared heads
    (2, 5, 130, 6, 2, 80),       # a beam
    (2, 41, 200, 2, 2, 64),
    (1, 130, 65, 3, 1, 40),      # just past a tile of queries, and of frames
    (2, 129, 257, 2, 1, 128),
    (2, 127, 383, 4, 4, 96),
    (1, 300, 1000, 4, 1, 64),
    (1, 128, 2500, 1, 1, 128),   # few rows, many frames
    (1, 9, 70, 2, 1, 5),         # widths no vector divides
    (1, 33, 70, 2, 2, 250),
]


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_whole(binding, record_margin, shape, dtype):
    _check(binding, shape, dtype, seed=1, record=record_margin, case="xattn whole %s" % str(dtype)[6:])


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] > 1] + [(5, 70, 300, 4, 2, 64)], ids=str)
def test_lengths_and_what_lies_past_them(binding, record_margin, shape, dtype):
    _check(binding, shape, dtype, seed=2, lens=True, record=record_margin, case="xattn lens %s" % str(dtype)[6:])


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(2, 41, 200, 2, 2, 64), (1, 300, 1000, 4, 1, 64), (2, 150, 257, 2, 1, 128),
                                   (3, 3, 500, 4, 2, 96), (1, 40, 90, 2, 2, 36)], ids=str)
@pytest.mark.parametrize("lens", [False, True])
def test_windows_some_empty(binding, record_margin, shape, dtype, lens):
    _check(binding, shape, dtype, seed=3, lens=lens, windows=True, record=record_margin,
           case="xattn windows %s" % str(dtype)[6:])


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
def test_other_layouts_scale_and_large_scores(binding, dtype):
    _check(binding, (2, 60, 150, 4, 2, 64), dtype, seed=4, fused=False)
    _check(binding, (2, 60, 150, 4, 2, 64), dtype, seed=5, scale=0.9)
    _check(binding, (2, 60, 400, 2, 2, 64), dtype, seed=6, std=6.0)   # scores of hundreds: one-hot softmax


def test_rows_that_no_vector_load_fits(binding):
    """Heads of a width and an offset that leave rows on odd addresses."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for dtype in TYPES:
        base = torch.randn(2, 100, 3, 67, generator=g, device="cuda").to(dtype)
        q, k, v = base[:, :20, :2, 1:65], base[:, :, :1, 2:66], base[:, :, 1:2, 3:67]
        go = base[:, 30:50, 1:3, 0:64]
        want = _reference(q, k, v, go, _seen(2, 20, 100, None, None, None, q.device), 0.125, dtype)
        out, lse = binding.tdt_cross_attn_fwd(q, k, v)
        dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse)
        for name, x in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
            _near(name, x, *want[name])


def test_broadcast_inputs_and_given_outputs(binding):
    """Frames shared by the batch (stride 0), results written into slices of wider tensors."""
    g = torch.Generator(device="cuda").manual_seed(4)
    dtype = torch.bfloat16
    q, go = (torch.randn(3, 50, 4, 64, generator=g, device="cuda").to(dtype) for _ in range(2))
    k, v = (torch.randn(1, 90, 2, 64, generator=g, device="cuda").to(dtype).expand(3, -1, -1, -1) for _ in range(2))
    want = _reference(q, k, v, go, _seen(3, 50, 90, None, None, None, q.device), 0.125, dtype)
    wide = torch.full((3, 50, 2, 4, 64), 7.0, dtype=dtype, device="cuda")
    dkv = torch.full((3, 90, 2, 2, 64), 7.0, dtype=dtype, device="cuda")
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, out=wide[:, :, 0])
    dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, dk=dkv[:, :, 0], dv=dkv[:, :, 1])
    assert dk.data_ptr() == dkv.data_ptr() and bool((wide[:, :, 1] == 7.0).all())
    for name, x in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
        _near(name, x, *want[name])


def test_no_frames_and_bad_lengths(binding):
    q, go = (torch.randn(2, 3, 2, 64, device="cuda") for _ in range(2))
    k = torch.empty(2, 0, 1, 64, device="cuda")
    out, lse = binding.tdt_cross_attn_fwd(q, k, k)
    dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, k, out, lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and bool((dq == 0).all())
    assert dk.shape == k.shape and dv.shape == k.shape
    for dtype in TYPES:
        q, go = (torch.randn(3, 9, 2, 64, device="cuda").to(dtype) for _ in range(2))
        k, v = (torch.randn(3, 30, 1, 64, device="cuda").to(dtype) for _ in range(2))
        for key, bad in (("k_lens", [31, -1, 30]), ("q_lens", [10, -2, 9])):
            a = {key: torch.tensor(bad, device="cuda")}
            out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
            assert bool(out[:2].isnan().all()) and bool(lse[:2].isnan().all())
            assert bool(out[2].isfinite().all())
            grads = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
            for x in grads:
                assert bool((x[:2] == 0).all()) and bool(x.isfinite().all())


def test_gradient_against_differences(binding):
    """The kernels' gradients along random directions against differences of the formula in 64 bits."""
    B, Lq, Lk, H, Hkv, D = shape = (2, 20, 60, 4, 2, 32)
    q, k, v, go, a = _inputs(shape, torch.float32, 9, lens=True, poison=False)
    seen = _seen(B, Lq, Lk, **a, dev=q.device)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
    grads = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)

    def value(q, k, v):
        return (_reference(q, k, v, go, seen, D ** -0.5, torch.float32)["out"][0] * go.double()).sum().item()

    x = [t.double() for t in (q, k, v)]
    g = torch.Generator(device="cuda").manual_seed(8)
    for n in range(3):
        d = torch.randn(x[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, down = ([t + s * h * d if i == n else t for i, t in enumerate(x)] for s in (1, -1))
        slope = (value(*up) - value(*down)) / (2 * h)
        mine = (grads[n].double() * d).sum().item()
        # differences err by h^2 times third derivatives of size one per element; the kernels by 1e-5 of the terms
        assert abs(mine - slope) <= 1e-5 * (grads[n].double() * d).abs().sum().item() + 1e-5


def test_same_inputs_same_bits(binding):
    for dtype in TYPES:
        q, k, v, go, a = _inputs((3, 140, 700, 4, 2, 64), dtype, 11, lens=True)
        runs = []
        for _ in range(3):
            out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
            runs.append((out, lse) + binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a))
        for other in runs[1:]:
            assert all(torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)) for x, y in zip(runs[0], other))


def test_on_another_stream_and_in_a_graph(binding):
    q, k, v, go, a = _inputs((2, 60, 300, 4, 4, 64), torch.bfloat16, 12, lens=True)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
    want = (out, lse) + binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, l2 = binding.tdt_cross_attn_fwd(q, k, v, **a)
        got = (o2, l2) + binding.tdt_cross_attn_bwd(go, q, k, v, o2, l2, **a)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = binding.tdt_cross_attn_fwd(q, k, v, **a)
        replayed = (o3, l3) + binding.tdt_cross_attn_bwd(go, q, k, v, o3, l3, **a)
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(want, got, replayed):
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)) and torch.equal(x.nan_to_num(7.0), z.nan_to_num(7.0))


def test_offsets_past_32_bits(binding):
    """Frames whose element offset does not fit 32 bits."""
    Lk, D = 70000, 64
    base = torch.zeros(2, Lk, 256 * D, dtype=torch.bfloat16, device="cuda")  # 1.15e9 elements an utterance
    frames = base.view(2, Lk, 256, D)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = frames[:, :, 254:255], frames[:, :, 255:256]
    k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
    v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
    for Lq in (1, 40):
        q, go = (torch.randn(2, Lq, 1, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        lo = torch.full((2, Lq), Lk - 200, dtype=torch.int32, device="cuda")
        w = torch.stack([lo, lo + 200], -1).contiguous()
        want = _reference(q, k[:, -200:], v[:, -200:], go, torch.ones(2, Lq, 200, dtype=torch.bool, device="cuda"),
                          0.125, torch.bfloat16)
        out, lse = binding.tdt_cross_attn_fwd(q, k, v, windows=w)
        _near("out", out, *want["out"])
        dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, windows=w)
        _near("dq", dq, *want["dq"])
        _near("dk", dk[:, -200:], *want["dk"])
        _near("dv", dv[:, -200:], *want["dv"])
        assert bool((dk[:, :-200] == 0).all()) and bool((dv[:, :-200] == 0).all())


@pytest.mark.parametrize("dtype", TYPES[1:], ids=["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_tails_of_every_walk_length(binding, dtype, D):
    """What lies past an utterance's end never shows, however many tiles come before the cut one."""
    for tiles in range(1, 13):
        for Lq in (40, 200):
            _check(binding, (1, Lq, tiles * 128 - 20, 1, 1, D), dtype, seed=tiles, lens=True)
            _check(binding, (1, tiles * 128 - 20, 150, 2, 1, D), dtype, seed=tiles, lens=True)


@pytest.mark.parametrize("lens,windows", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("shape", [(1, 9, 1, 1, 1, 65), (1, 20, 130, 1, 1, 128), (2, 129, 500, 2, 2, 80), (1, 50, 5000, 2, 1, 68),
                                   (2, 100, 260, 8, 2, 96), (1, 700, 300, 6, 2, 128), (3, 300, 1100, 16, 1, 72)], ids=str)
def test_float32_heads_over_64(binding, record_margin, shape, lens, windows):
    """One tile and many, walks shared by 1 to 8 blocks, packed heads, widths that fill their last part or not."""
    _check(binding, shape, torch.float32, record=record_margin, case=f"wide {shape}", lens=lens, windows=windows)


def test_float32_heads_over_64_off_the_usual_ways(binding):
    """Odd addresses, bad lengths, another stream, a graph, and the same bits each time."""
    g = torch.Generator(device="cuda").manual_seed(13)
    base = torch.randn(2, 300, 3, 99, generator=g, device="cuda")
    q, k, v, go = base[:, :70, :2, 1:97], base[:, :, :1, 2:98], base[:, :, 1:2, 3:99], base[:, 80:150, 1:3, 0:96]
    want = _reference(q, k, v, go, _seen(2, 70, 300, None, None, None, q.device), 96 ** -0.5, torch.float32)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v)
    dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse)
    for name, x in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
        _near(name, x, *want[name])
    q, go = (torch.randn(3, 70, 2, 96, generator=g, device="cuda") for _ in range(2))
    k, v = (torch.randn(3, 130, 1, 96, generator=g, device="cuda") for _ in range(2))
    for key, bad in (("k_lens", [131, -1, 130]), ("q_lens", [71, -2, 70])):
        a = {key: torch.tensor(bad, device="cuda")}
        out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
        assert bool(out[:2].isnan().all()) and bool(lse[:2].isnan().all()) and bool(out[2].isfinite().all())
        for x in binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a):
            assert bool((x[:2] == 0).all()) and bool(x.isfinite().all())
    q, k, v, go, a = _inputs((3, 140, 1500, 4, 2, 128), torch.float32, 14, lens=True, windows=True)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
    want = (out, lse) + binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, l2 = binding.tdt_cross_attn_fwd(q, k, v, **a)
        got = (o2, l2) + binding.tdt_cross_attn_bwd(go, q, k, v, o2, l2, **a)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = binding.tdt_cross_attn_fwd(q, k, v, **a)
        replayed = (o3, l3) + binding.tdt_cross_attn_bwd(go, q, k, v, o3, l3, **a)
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(want, got, replayed):
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)) and torch.equal(x.nan_to_num(7.0), z.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(2, 9, 300, 2, 2, 64), (2, 5, 200, 12, 4, 40), (1, 32, 130, 1, 1, 128), (2, 3, 90, 8, 1, 192),
                                   (1, 33, 130, 1, 1, 72), (2, 11, 500, 6, 2, 256)], ids=str)
def test_rows_shared_by_blocks(binding, record_margin, shape, dtype):
    """9 to 33 rows a key head: several blocks share a key head's rows, the last one in part."""
    for how in (dict(), dict(lens=True), dict(lens=True, windows=True)):
        _check(binding, shape, dtype, record=record_margin, case=f"rows {shape}", **how)


def _past_lengths(shape, dtype, q_len, k_len, past, seed=0, empty=None):
    """Inputs of one head width whose rows and frames past the lengths hold `past`; rows of `empty` have empty windows."""
    B, Lq, Lk, H, Hkv, D = shape
    q, k, v, go, a = _inputs(shape, dtype, seed, lens=True, poison=False)
    a["q_lens"].fill_(q_len)
    a["k_lens"].fill_(k_len)
    for t, n in ((q, q_len), (go, q_len), (k, k_len), (v, k_len)):
        t[:, n:] = past
    if empty:
        w = torch.zeros(B, Lq, 2, dtype=torch.int32, device="cuda")
        w[..., 1] = Lk
        w[:, slice(*empty)] = 0
        a["windows"] = w
    return q, k, v, go, a


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("past", [math.nan, math.inf], ids=["nan", "inf"])
@pytest.mark.parametrize("Lk,k_len", [(200, 100), (2000, 1900)])  # one block a walk, and several
@pytest.mark.parametrize("H,Lq,q_lens", [(2, 121, (0, 1, 31, 32, 33, 60, 64, 121)), (4, 31, (0, 8, 15, 31))])
def test_rows_that_take_no_part_beside_frames_that_hold_anything(binding, dtype, past, Lk, k_len, H, Lq, q_lens):
    """Whole warps of rows past the queries' length, in tiles whose frames past theirs are no numbers."""
    for q_len in q_lens:
        q, k, v, go, a = _past_lengths((1, Lq, Lk, H, 2, 64), dtype, q_len, k_len, past)
        want = _reference(q, k, v, go, _seen(1, Lq, Lk, **a, dev=q.device), 0.125, dtype)
        out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
        dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
        assert bool((dq[:, q_len:] == 0).all()), q_len
        for name, x in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
            _near(name, x, *want[name])


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("Lq", [121, 300])  # one row tile and three
def test_empty_windows_beside_frames_that_hold_anything(binding, dtype, Lq):
    q, k, v, go, a = _past_lengths((2, Lq, 200, 2, 2, 64), dtype, Lq, 100, math.nan, empty=(32, 64))
    want = _reference(q, k, v, go, _seen(2, Lq, 200, **a, dev=q.device), 0.125, dtype)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
    dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
    assert bool((dq[:, 32:64] == 0).all())
    for name, x in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
        _near(name, x, *want[name])


def _norm_errors(binding, q, k, v, go, a, dtype, units, least=None):
    """The results' errors in 2-norm, each of its value's norm times `units` plus what the type's least step makes of it."""
    D = q.shape[3]
    want = _reference(q, k, v, go, _seen(q.shape[0], q.shape[1], k.shape[1], **a, dev=q.device), D ** -0.5, dtype)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
    dq, dk, dv = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
    for name, x in dict(out=out, dq=dq, dk=dk, dv=dv).items():
        value = want[name][0]
        bound = units * value.norm().item() + (least or 0.0) / 2 * value.numel() ** 0.5
        error = (x.double() - value).norm().item()
        assert error <= bound, "%s: %.3g of its norm, %.3g allowed" % (
            name, error / value.norm().item(), bound / value.norm().item())


F16_SHAPES = [(1, 121, 2000, 2, 2, 64), (1, 300, 2000, 2, 2, 64), (2, 300, 700, 4, 2, 96), (3, 30, 500, 8, 2, 40)]


@pytest.mark.parametrize("std", [1.0, 1e-3, 3e-4, 1e-4, 1e-5])
@pytest.mark.parametrize("shape", F16_SHAPES, ids=str)
def test_float16_small_upstream_gradients(binding, shape, std):
    """Gradients keep the type's accuracy where grad_out times a weight is below the type's normal range.

    Bound: a unit each for the results' rounding, for that of dS (or P) and for delta's from the rounded out; and half
    a least step of the type an element."""
    q, k, v, go, a = _inputs(shape, torch.float16, 21, lens=shape[0] > 1)
    _norm_errors(binding, q, k, v, go * std, a, torch.float16, 3 * UNIT[torch.float16], 2.0 ** -24)


@pytest.mark.parametrize("Lq", [100, 300])
def test_float16_large_upstream_gradients(binding, Lq):
    """grad_out . v past the type's range, results within it: nothing overflows on the way."""
    q, k, v, go, a = _inputs((2, Lq, 8, 2, 2, 64), torch.float16, 22)
    _norm_errors(binding, q * 0.05, k * 0.25, v * 16.0, go * 4000.0, a, torch.float16, 3 * UNIT[torch.float16], 2.0 ** -24)


def test_float16_utterances_of_other_sizes(binding):
    """Each utterance and key head has its own range: one of grad_out 1e4 beside one of 1e-4, zeros beside both."""
    for Lq in (60, 200):
        q, k, v, go, a = _inputs((3, Lq, 900, 4, 2, 64), torch.float16, 23)
        go[0] *= 1e3
        go[1] *= 1e-4
        go[2] = 0.0
        out, lse = binding.tdt_cross_attn_fwd(q, k, v)
        for x in binding.tdt_cross_attn_bwd(go, q, k, v, out, lse):
            assert bool((x[2] == 0).all())
        for b in (0, 1):
            _norm_errors(binding, *(t[b:b + 1] for t in (q, k, v, go)), a, torch.float16, 3 * UNIT[torch.float16], 2.0 ** -24)
        want = [binding.tdt_cross_attn_bwd(*(t[b:b + 1] for t in (go, q, k, v, out)), lse[b:b + 1].contiguous())
                for b in (0, 1)]
        got = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse)
        for b in (0, 1):
            for x, y in zip(got, want[b]):
                assert (x[b:b + 1].double() - y.double()).norm() <= 2 * UNIT[torch.float16] * y.double().norm() + 1e-7 * y.numel() ** 0.5


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(2, 121, 2500, 2, 2, 64), (2, 300, 1000, 4, 2, 64), (1, 130, 2500, 2, 1, 128),
                                   (2, 3, 1500, 4, 2, 96), (4, 1, 2000, 4, 4, 64), (1, 40, 1000, 2, 1, 200)], ids=str)
def test_errors_in_norm(binding, shape, dtype):
    """Three units of the type (results, P or dS, delta) in 2-norm; float32: exponentials good to 2^-20, four times
    that.  One average frame of 2,500 that is missing or doubled changes the results by 2 %."""
    units = 3 * UNIT[dtype] if dtype != torch.float32 else 2.0 ** -18
    q, k, v, go, a = _inputs(shape, dtype, 24, lens=shape[0] > 1)
    _norm_errors(binding, q, k, v, go, a, dtype, units, 2.0 ** -24 if dtype == torch.float16 else None)


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
def test_given_workspace(binding, dtype):
    for shape in ((2, 70, 900, 4, 2, 64), (1, 300, 700, 2, 1, 96), (1, 10, 300, 2, 1, 200)):
        q, k, v, go, a = _inputs(shape, dtype, 25, lens=True)
        ws = [torch.full((binding.tdt_cross_attn_workspace_size(shape, dtype, back) + 1,), 255, dtype=torch.uint8, device="cuda")
              for back in (False, True)]
        out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
        o2, l2 = binding.tdt_cross_attn_fwd(q, k, v, workspace=ws[0], **a)
        grads = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
        g2 = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, workspace=ws[1], **a)
        for x, y in zip((out, lse) + grads, (o2, l2) + g2):
            assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))
        assert ws[0][-1] == 255 and ws[1][-1] == 255


@pytest.mark.parametrize("dtype", TYPES[1:], ids=["f16", "bf16"])
@pytest.mark.parametrize("Lk,windows", [(20, 0), (40, 0), (60, 0), (128, 0), (130, 0), (200, 0), (256, 0), (900, 30), (900, 200)])
@pytest.mark.parametrize("shape", [(4, 60, 8, 8, 64), (3, 150, 4, 2, 128), (2, 200, 6, 2, 40)], ids=str)
def test_gradients_where_rows_see_few_frames(binding, dtype, shape, Lk, windows):
    """Two roundings to 16 bits, of dS and of the results, and no third one of delta.

    A rounding to nearest errs by 0.43 units in norm (a third of a squared half step, over the mantissas of a binade), two by
    0.61; 0.65 leaves the sample's scatter."""
    B, Lq, H, Hkv, D = shape
    q, k, v, go, a = _inputs((B, Lq, Lk, H, Hkv, D), dtype, 26, std=1.0)
    if windows:
        at = torch.arange(Lq, device="cuda") * (Lk - windows) // Lq
        a["windows"] = torch.stack([at, at + windows], -1).to(torch.int32).expand(B, -1, -1).contiguous()
    want = _reference(q, k, v, go, _seen(B, Lq, Lk, **a, dev=q.device), D ** -0.5, dtype)
    out, lse = binding.tdt_cross_attn_fwd(q, k, v, **a)
    dq, dk, _ = binding.tdt_cross_attn_bwd(go, q, k, v, out, lse, **a)
    for name, x in (("dq", dq), ("dk", dk)):
        value = want[name][0]
        error = ((x.double() - value).norm() / value.norm()).item()
        assert error <= 0.65 * UNIT[dtype], "%s: %.3g of its norm, %.3g allowed" % (name, error, 0.65 * UNIT[dtype])
