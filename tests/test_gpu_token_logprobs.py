"""Log-probabilities of given tokens, entropies, alternatives and gradients on the GPU against the formulas in 64 bits.

Tolerances count roundings: logits enter exactly, z = x - max is rounded once (2^-24 |z|), exponentials are good to 2^-20 and to the
rounding of z log2(e), sums of V positive terms of float32 to (V^0.5 + 30) 2^-24 in any order of halves, results once; gradients once
more to their own type (unit u).
"""
import math

import pytest
import torch

from paged_cases import TYPES, UNIT

pytestmark = pytest.mark.gpu
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transducer_loss_asr_gb300 import binding as b

    return b


def _reference(x, tokens, n_top, a=None, b=None, c=None):
    """{name: (value, bound)} in 64 bits for rows that all take part."""
    N, V = x.shape
    dtype, e32 = x.dtype, 2.0 ** -24
    x = x.double()
    m = x.amax(1, keepdim=True)
    z = x - m
    zs = torch.where(z < -1e4, 0.0, z)  # weight 0
    ez = e32 * zs.abs() * 3 + 2.0 ** -20                 # relative error of a weight
    w = torch.exp(z)
    s = w.sum(1, keepdim=True)
    sums = (V ** 0.5 + 30) * e32
    es = (w * ez).sum(1, keepdim=True) / s + sums        # of their sum
    ln_s = torch.log(s)
    e_ln = es + 2.0 ** -20 + 2 * e32 * ln_s.abs()        # log2's own error, and ln 2
    lp = z - ln_s
    e_lp = e32 * 2 * (torch.where(z.isinf(), 0.0, z).abs() + ln_s) + e_ln
    p = w / s
    plp = torch.where(p > 0, p * torch.where(lp < -1e4, 0.0, lp), 0.0)
    ent = -plp.sum(1)
    e_ent = (p * zs.abs() * (ez + es + sums)).sum(1) + e_ln[:, 0] + 4 * e32 * (ent + ln_s[:, 0])
    at = tokens[:, None]
    r = dict(logprobs=(lp.gather(1, at)[:, 0], e_lp.gather(1, at)[:, 0] + 1e-30), entropy=(ent, e_ent + 1e-30))
    if n_top:
        top = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :n_top]
        r["top_tokens"] = top
        r["top_logprobs"] = (lp.gather(1, top), e_lp.gather(1, top) + 1e-30)
    if a is not None or b is not None or c is not None:
        zero = torch.zeros(N, dtype=torch.float64, device=x.device)
        a, b = (zero if t is None else t.double() for t in (a, b))
        total = a if c is None else a + c.double().sum(1)
        lpf = torch.where(lp < -1e4, 0.0, lp)
        d = -p * total[:, None] - b[:, None] * (plp + p * ent[:, None])
        d.scatter_add_(1, at, a[:, None])
        own = torch.zeros_like(d).scatter_add_(1, at, a.abs()[:, None])
        if c is not None:
            d.scatter_add_(1, r["top_tokens"], c.double())
            own.scatter_add_(1, r["top_tokens"], c.double().abs())
        size = total.abs()[:, None] + b.abs()[:, None] * (lpf.abs() + ent[:, None])
        if c is not None:
            size = size + c.double().abs().sum(1)[:, None] * n_top * e32
        ep = e_lp + 2.0 ** -20 + 3 * e32 * lpf.abs()
        tol = p * size * (ep + 8 * e32) + p * b.abs()[:, None] * (e_lp + e_ent[:, None]) + 4 * e32 * own + UNIT[dtype] * d.abs()
        r["grad"] = (d, tol + TINY[dtype] * (1 + size))
    return r


def _near(name, x, want, record=None, case=""):
    if not isinstance(want, tuple):
        assert torch.equal(x.long(), want), name
        return
    value, bound = want
    x = x.double()
    same = torch.equal(x.isinf(), value.isinf()) and torch.equal(x.isnan(), value.isnan())
    assert same, name
    fine = value.isfinite()
    ratio = ((x - value).abs()[fine] / bound[fine]).max().item()
    if record:
        record(case, name, ratio, 1.0)
    assert ratio <= 1.0, "%s: error is %.3g of its bound" % (name, ratio)


def _inputs(N, V, dtype, seed, std=3.0, off=0, width=None, whole=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, width or V + 2 * off, generator=g, device="cuda") * std
    if whole:
        x = torch.round(x)  # ties are common
    x = x.to(dtype)[:, off:off + V]
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
    a, b = torch.randn(2, N, generator=g, device="cuda").unbind(0)
    return x, tokens, a.contiguous(), b.contiguous(), g


def _check(binding, x, tokens, n_top, a, b, g, record=None, case=""):
    N, V = x.shape
    c = torch.randn(N, n_top, generator=g, device="cuda") if n_top else None
    r = binding.tdt_token_logprobs_fwd(x, tokens, n_top)
    grad = binding.tdt_token_logprobs_bwd(x, tokens, r, a, b, c)
    want = _reference(x, tokens, n_top, a, b, c)
    for name, w in want.items():
        _near(name, grad if name == "grad" else getattr(r, name), w, record, case)
    r2, grad2 = binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b, n_top)
    want = _reference(x, tokens, n_top, a, b)
    _near("grad", grad2, want["grad"], record, case + " one call")
    for name in ("logprobs", "entropy", "top_tokens", "top_logprobs"):
        if name in want:
            _near(name, getattr(r2, name), want[name])
    lse = r.stats.double().sum(1)
    assert bool(((lse - torch.logsumexp(x.double(), 1)).abs() <= 1e-5 * (1 + lse.abs())).all())


SIZES = [(1, 1, 0), (1, 1, 1), (3, 2, 2), (5, 7, 3), (40, 33, 10), (7, 100, 64), (64, 1000, 20), (20, 8193, 10), (3, 8193, 64), (9, 50257, 20),
         (1, 131072, 32), (2, 140001, 5), (300, 257, 1)]


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V,n_top", SIZES)
def test_whole(binding, record_margin, N, V, n_top, dtype):
    x, tokens, a, b, g = _inputs(N, V, dtype, N + V)
    _check(binding, x, tokens, n_top, a, b, g, record_margin, "logprobs %s" % str(dtype)[6:])


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V,n_top", [(609, 10239, 20), (608, 10239, 5), (610, 10241, 64), (609, 20479, 3), (609, 20481, 0), (700, 2000, 64), (613, 4695, 32)])
def test_many_rows(binding, N, V, n_top, dtype):
    """Rows that are more than fit at once, on both sides of 40 KB; equal logits, and rows that hold one value."""
    x, tokens, a, b, g = _inputs(N, V, dtype, N + V, off=1)
    x[1::7] = torch.round(x[1::7])
    x[2::31] = 1.5
    _check(binding, x, tokens, n_top, a, b, g)


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V,n_top", [(4, 5, 3), (6, 1000, 64), (5, 8193, 33), (3, 50257, 20)])
def test_ties(binding, N, V, n_top, dtype):
    """Whole numbers: equal logits are everywhere, and alternatives come by rising token."""
    for std in (3.0, 0.3, 0.0):
        x, tokens, a, b, g = _inputs(N, V, dtype, V, std=std, whole=True)
        _check(binding, x, tokens, n_top, a, b, g)


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [300, 8193, 60000])
def test_sorted_and_clustered_rows(binding, V, dtype):
    """Rows that rise, fall, or hold their largest entries side by side or at one stride."""
    x = torch.zeros(8, V, device="cuda")
    ramp = torch.linspace(-8, 8, V, device="cuda")
    x[0], x[1], x[2], x[3] = ramp, -ramp, ramp.abs(), -ramp.abs()
    x[4, V // 2:V // 2 + 200] = 5.0 + torch.arange(min(200, V - V // 2), device="cuda") / 50.0
    x[5, ::256] = 4.0 + torch.arange(len(x[5, ::256]), device="cuda") / 64.0
    x[6, ::8] = 4.0
    x[7] = torch.where(torch.arange(V, device="cuda") < 40, 3.0, -5.0)
    tokens = torch.randint(0, V, (8,), device="cuda")
    a, b = torch.randn(2, 8, device="cuda").unbind(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    for n_top in (1, 20, 64):
        _check(binding, x.to(dtype), tokens, n_top, a.contiguous(), b.contiguous(), g)


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("std,mean", [(30.0, 0.0), (0.01, 0.0), (3.0, 1000.0), (3.0, -1000.0)])
def test_other_sizes_of_logits(binding, dtype, std, mean):
    x, tokens, a, b, g = _inputs(16, 5000, dtype, 3, std=std)
    _check(binding, (x.float() + mean).to(dtype), tokens, 10, a, b, g)


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
def test_slices_in_place_and_given_gradients(binding, dtype):
    """Rows of a wider tensor on any address; the gradient over the logits, or into a slice."""
    for V, off in ((8193, 0), (8193, 3), (1000, 1), (50257, 5)):
        x, tokens, a, b, g = _inputs(6, V, dtype, off, off=off, width=V + 13)
        _check(binding, x, tokens, 5, a, b, g)
        r = binding.tdt_token_logprobs_fwd(x, tokens)
        want = binding.tdt_token_logprobs_bwd(x, tokens, r, a, b)
        wide = torch.full((6, V + 9), 7.0, dtype=dtype, device="cuda")
        got = binding.tdt_token_logprobs_bwd(x, tokens, r, a, b, grad_out=wide[:, 2:V + 2])
        assert torch.equal(got, want) and bool((wide[:, :2] == 7.0).all()) and bool((wide[:, V + 2:] == 7.0).all())
        one = binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b)[1]
        for over in ("split", "one"):
            base = torch.full((6, V + 13), 7.0, dtype=dtype, device="cuda")
            y = base[:, off:off + V]
            y.copy_(x)
            if over == "split":
                got = binding.tdt_token_logprobs_bwd(y, tokens, r, a, b, grad_out=y)
                assert torch.equal(got, want)
            else:
                r2, got = binding.tdt_token_logprobs_fwd_bwd(y, tokens, a, b, grad_out=y)
                assert torch.equal(got, one) and torch.equal(r2.logprobs, r.logprobs)
            assert got.data_ptr() == y.data_ptr()
            assert bool((base[:, :off] == 7.0).all()) and bool((base[:, off + V:] == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [50, 8193, 40000])
def test_padding_tokens_out_of_range_and_masked_entries(binding, dtype, V):
    N, K = 12, 8
    x, tokens, a, b, g = _inputs(N, V, dtype, 7)
    x[4, ::2] = -math.inf          # tokens that are not allowed
    x[5] = -math.inf               # all but one
    x[5, 17] = 2.0
    tokens[4], tokens[5] = 1, 17
    tokens[6] = 2                  # a token that is not allowed
    x[6, 2] = -math.inf
    tokens[:4] = torch.tensor([-100, -1, V, 2 ** 40], device="cuda")
    x[0], x[1] = math.nan, math.inf  # not read
    x[7, 3] = math.nan
    x[8, 4] = math.inf
    x[9] = -math.inf
    r = binding.tdt_token_logprobs_fwd(x, tokens, K)
    grad = binding.tdt_token_logprobs_bwd(x, tokens, r, a, b)
    r2, grad2 = binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b, K)
    for q, d in ((r, grad), (r2, grad2)):
        assert bool((q.logprobs[:2] == 0).all()) and bool((q.entropy[:2] == 0).all()) and bool((q.stats[:2] == 0).all())
        assert bool((q.top_tokens[:4] == -1).all()) and bool((q.top_logprobs[:2] == -math.inf).all())
        assert bool(q.logprobs[2:4].isnan().all()) and bool(q.entropy[2:4].isnan().all()) and bool(q.top_logprobs[2:4].isnan().all())
        assert bool((d[:4] == 0).all())
        for i in (7, 8, 9):
            assert bool(q.logprobs[i].isnan()) and bool(q.entropy[i].isnan())
            assert bool((q.top_tokens[i] == -1).all()) and bool(q.top_logprobs[i].isnan().all()) and bool(d[i].isnan().all())
        rows = torch.tensor([4, 5, 6, 10, 11], device="cuda")
        want = _reference(x[rows], tokens[rows], K, a[rows], b[rows])
        for name, w in want.items():
            _near(name, (d if name == "grad" else getattr(q, name))[rows], w)
        assert float(q.logprobs[6]) == -math.inf


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [30, 700, 8193, 50257])
def test_masks_of_the_types_lowest_value_and_few_allowed_tokens(binding, V, dtype):
    """Most entries are -inf or the type's lowest number; fewer tokens than alternatives are allowed."""
    N, K = 6, 20
    x, tokens, a, b, g = _inputs(N, V, dtype, 11)
    low = torch.finfo(dtype).min
    few = torch.randint(0, V, (N, 7), generator=g, device="cuda")
    mask = torch.ones(N, V, dtype=torch.bool, device="cuda").scatter_(1, few, False)
    x[0] = torch.where(mask[0], -math.inf, x[0])
    x[1] = torch.where(mask[1], low, x[1])
    x[2] = torch.where(mask[2], torch.where(torch.arange(V, device="cuda") % 2 == 0, low, -math.inf).to(dtype), x[2])
    x[3, :V // 2] = low            # what a thread sees first
    x[4, :V // 2] = -math.inf
    x[5] = torch.where(torch.arange(V, device="cuda") % 3 == 0, low, -math.inf).to(dtype)  # uniform over a third
    tokens[:3], tokens[3:] = few[:3, 0], V - V % 3 - 3
    x[3:5, V - V % 3 - 3] = 1.0
    _check(binding, x, tokens, K, a, b, g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [30, 700, 8193, 50257])
def test_logits_at_the_ends_of_the_range(binding, V, dtype):
    """Products with log2 e of such logits, or their differences, leave float32's range; p and the entropy do not."""
    N = 10
    x, tokens, a, b, g = _inputs(N, V, dtype, 13)
    low = torch.finfo(dtype).min
    x[0], x[1], x[2] = -math.inf, low, -(2.0 ** 126)
    x[3] = x[3].float() * 1e37
    x[4] = torch.where(torch.arange(V, device="cuda") % 2 == 0, low, -math.inf).to(dtype)
    x[5], x[6], x[7] = low, -math.inf, low
    x[8], x[9] = -1.5e38, -math.inf
    for i, top in enumerate((2.0 ** 126, 2.0 ** 126, 2.0 ** 126, 1.75 * 2.0 ** 126, 2.0 ** 100, 2.0 ** 127, -(2.0 ** 126), -(2.0 ** 126), 1e38, -1.5e38)):
        x[i, V // 3] = x[i, V // 2 + 1] = x[i, V - 1] = top  # an entropy of ln 3
    tokens[:] = V // 2 + 1
    _check(binding, x, tokens, 3, a, b, g)
    assert torch.allclose(binding.tdt_token_logprobs_fwd(x, tokens).entropy.cpu(), torch.full((N,), math.log(3.0)), atol=1e-5, rtol=0)


def test_missing_weights(binding):
    x, tokens, a, b, g = _inputs(5, 700, torch.float32, 3)
    r = binding.tdt_token_logprobs_fwd(x, tokens, 4)
    c = torch.randn(5, 4, device="cuda")
    for aa, bb, cc in ((a, None, None), (None, b, None), (None, None, c), (None, b, c)):
        _near("grad", binding.tdt_token_logprobs_bwd(x, tokens, r, aa, bb, cc), _reference(x, tokens, 4, aa, bb, cc)["grad"])
    assert bool((binding.tdt_token_logprobs_bwd(x, tokens, r) == 0).all())
    assert bool((binding.tdt_token_logprobs_fwd_bwd(x, tokens)[1] == 0).all())


def test_same_inputs_same_bits_streams_and_graphs(binding):
    for dtype in TYPES:
        for N, V in ((1, 50257), (30, 8193), (400, 3000)):
            x, tokens, a, b, g = _inputs(N, V, dtype, 5)
            want = (*binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b, 6)[0], binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b, 6)[1])
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                r, d = binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b, 6)
            torch.cuda.current_stream().wait_stream(s)
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                r2, d2 = binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b, 6)
            for _ in range(2):
                graph.replay()
            for p, q, t in zip(want, (*r, d), (*r2, d2)):
                assert torch.equal(p, q) and torch.equal(p, t)


def test_rows_past_32_bits(binding):
    """A tensor of more than 2^31 elements, and rows far apart."""
    N, V = 20, 300
    base = torch.zeros(N, 2 ** 27, dtype=torch.bfloat16, device="cuda")
    x, tokens, a, b, g = _inputs(N, V, torch.bfloat16, 5)
    y = base[:, -V:]
    y.copy_(x)
    r = binding.tdt_token_logprobs_fwd(y, tokens, 3)
    for name, w in _reference(x, tokens, 3).items():
        _near(name, getattr(r, name), w)
    grad = binding.tdt_token_logprobs_bwd(x, tokens, r, a, b)
    binding.tdt_token_logprobs_bwd(y, tokens, r, a, b, grad_out=y)
    assert torch.equal(y, grad) and bool((base[:, :-V] == 0).all())


def test_autograd_against_the_formula_and_differences(binding):
    """Through a strided view of joint outputs, with padded labels; all three results weighted."""
    from transducer_loss_asr_gb300 import autograd

    g = torch.Generator(device="cuda").manual_seed(4)
    base = torch.randn(2, 5, 3, 60, generator=g, device="cuda")
    tokens = torch.randint(0, 50, (2, 5, 3), generator=g, device="cuda")
    tokens[0, 3:] = -100
    w = torch.randn(2, 5, 3, 6, generator=g, device="cuda").double()
    real = (tokens >= 0).double()

    def formula(x):
        lp = torch.log_softmax(x[..., :50], -1)
        ent = -(lp.exp() * lp).sum(-1)
        top = lp.topk(4, -1).values
        given = lp.gather(-1, tokens.clamp_min(0)[..., None])[..., 0]
        return (real * (w[..., 0] * given + w[..., 1] * ent + (w[..., 2:] * top).sum(-1))).sum()

    x = base.clone().requires_grad_()
    lp, ent, top, top_lp = autograd.TokenLogprobs()(x[..., :50], tokens, 4)
    assert lp.shape == tokens.shape and top.shape == (2, 5, 3, 4) and not top.requires_grad
    top_lp = torch.where(tokens[..., None] >= 0, top_lp, 0.0)
    (w[..., 0] * lp + w[..., 1] * ent + (w[..., 2:] * top_lp).sum(-1)).sum().backward()
    x64 = base.double().requires_grad_()
    formula(x64).backward()
    # weights of size 1, six terms: float32 roundings of each
    assert bool(((x.grad.double() - x64.grad).abs() <= 2e-5).all())
    for n in range(3):
        d = torch.randn(base.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        slope = (formula(base.double() + h * d) - formula(base.double() - h * d)) / (2 * h)
        mine = (x.grad.double() * d).sum()
        # differences err by h^2 times third derivatives and 1e-16 / h
        assert abs(float(mine - slope)) <= 2e-5 * float((x.grad.double() * d).abs().sum()) + 1e-6


def test_tokens_that_are_slices(binding):
    from transducer_loss_asr_gb300.autograd import token_logprobs

    x, tokens, *_ = _inputs(12, 50, torch.float32, 3)
    want = token_logprobs(x, tokens)[0]
    wide = torch.stack((tokens, tokens + 1), 1)
    assert torch.equal(token_logprobs(x, wide[:, 0])[0], want)
    assert torch.equal(token_logprobs(x.view(3, 4, 50), wide.view(3, 4, 2)[..., 0])[0], want.view(3, 4))
    assert torch.equal(token_logprobs(x.view(3, 4, 50).transpose(0, 1), tokens.view(3, 4).t())[0], want.view(3, 4).t())


def test_compiled_opcheck_and_a_captured_backward(binding):
    from transducer_loss_asr_gb300 import autograd

    x, tokens, a, b, g = _inputs(12, 500, torch.bfloat16, 9)
    x = x.contiguous().requires_grad_()
    m = autograd.TokenLogprobs()

    def loss(f):
        lp, ent, _, top = f(x, tokens, 3)
        return -(a * lp).sum() - 0.1 * ent.sum() + top.sum()

    want = torch.autograd.grad(loss(m), x)[0]
    got = torch.autograd.grad(loss(torch.compile(m, fullgraph=True)), x)[0]
    assert torch.equal(want, got)
    only = torch.autograd.grad(m(x, tokens)[1].sum(), x)[0]  # the entropy alone
    assert bool(only.isfinite().all()) and float(only.abs().sum()) > 0
    torch.library.opcheck(torch.ops.tdt_gb300.token_logprobs_forward.default, (x.detach(), tokens, 3),
                          test_utils=("test_schema", "test_faketensor"))
    torch.library.opcheck(torch.ops.tdt_gb300.token_logprobs_forward.default, (x.detach(), tokens, 0),
                          test_utils=("test_schema", "test_faketensor"))


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V", [(12, 60), (6, 700), (7, 8193), (5, 50257), (700, 4000), (1, 300000)])
def test_entropy_weights_of_any_size_over_masked_tokens(binding, N, V, dtype):
    """-inf or the type's lowest number here and there: such an entry's gradient is 0, however large the entropy's weight.  Both
    calls, over the logits, and into rows on another address."""
    x, tokens, a, b, g = _inputs(N, V, dtype, 17)
    mask = torch.randint(0, 16, (N, V), generator=g, device="cuda") == 0
    mask.scatter_(1, tokens[:, None], False)
    x = torch.where(mask, -math.inf, x)
    x[1::2] = x[1::2].clamp_min(torch.finfo(dtype).min)
    # float16 results end at 65504; entropies here are under 12, so that products with them stay in float32
    sizes = [2.0, -2.0, 100.0, -50.0, 1.75] if dtype == torch.float16 else [2.0, -2.0, 65536.0, -1e20, 1e37]
    for turn in range(len(sizes) if N < len(sizes) else 1):
        b = torch.tensor(sizes[turn:] + sizes[:turn], device="cuda").repeat(N // len(sizes) + 1)[:N].contiguous()
        _check(binding, x, tokens, 0, a, b, g)
        r = binding.tdt_token_logprobs_fwd(x, tokens)
        split = binding.tdt_token_logprobs_bwd(x, tokens, r, a, b)
        one = binding.tdt_token_logprobs_fwd_bwd(x, tokens, a, b)[1]
        assert bool((split[mask] == 0).all()) and bool((one[mask] == 0).all())
        for off in (0, 3):
            wide = torch.empty(N, V + 8, dtype=dtype, device="cuda")[:, off:off + V]
            assert torch.equal(binding.tdt_token_logprobs_bwd(x, tokens, r, a, b, grad_out=wide), split)
            base = torch.zeros(N, V + 8, dtype=dtype, device="cuda")
            y = base[:, off:off + V].copy_(x)
            assert torch.equal(binding.tdt_token_logprobs_bwd(y, tokens, r, a, b, grad_out=y), split)
            y.copy_(x)
            got = binding.tdt_token_logprobs_fwd_bwd(y, tokens, a, b, grad_out=y)[1]
            assert bool((got[mask] == 0).all()) and bool(got.isfinite().all())


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V", [(40, 700), (12, 8193), (9, 60000), (1, 131072), (700, 4000)])
def test_stretches_of_masked_tokens_weigh_nothing(binding, N, V, dtype):
    """What a thread, a warp or a CTA sees first, or all that it sees, is masked: its sums are nothing, and results are, bit for
    bit, those over logits so far below the others that their weight is 0."""
    x, _, a, b, g = _inputs(N, V, dtype, 19)
    at = torch.arange(V, device="cuda")
    few = torch.zeros(V, dtype=torch.bool, device="cuda")
    few[torch.randperm(V, generator=g, device="cuda")[:7]] = True
    lowest = [-math.inf, torch.finfo(dtype).min] + ([] if dtype == torch.float16 else [-1e30])
    for allowed in (at >= V // 2, at < V // 10, (at >= V // 3) & (at < V // 2), few):
        ids = allowed.nonzero()[:, 0]
        tokens = ids[torch.randint(0, len(ids), (N,), generator=g, device="cuda")]
        far = torch.where(allowed, x, -1e4)
        want, want_grad = binding.tdt_token_logprobs_fwd_bwd(far, tokens, a, b, 5)
        scores = binding.tdt_token_logprobs_fwd(far, tokens, 5)
        for low in lowest:
            y = torch.where(allowed, x, low)
            got, grad = binding.tdt_token_logprobs_fwd_bwd(y, tokens, a, b, 5)
            for p, q in zip((*want, want_grad, *scores), (*got, grad, *binding.tdt_token_logprobs_fwd(y, tokens, 5))):
                assert torch.equal(p, q), low


@pytest.mark.parametrize("V", [40, 700, 8193, 60000])
def test_maxima_on_both_sides_of_the_largest_reference(binding, V):
    """float32 logits near +-2^24 / log2(e), where the reference of a row gives way to its maximum; masked tokens beside them."""
    edge = 2.0 ** 24 / math.log2(math.e)
    x, tokens, a, b, g = _inputs(12, V, torch.float32, 23)
    base = torch.tensor([s * (edge + d) for s in (1.0, -1.0) for d in (-200.0, -12.0, -3.0, 0.0, 7.0, 300.0)], device="cuda")
    x = torch.round(x * 2) + base[:, None]
    x[1::2, :V // 2] = -math.inf
    tokens = torch.randint(V // 2, V, (12,), generator=g, device="cuda")
    _check(binding, x, tokens, 5, a, b, g)
