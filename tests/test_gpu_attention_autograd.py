"""Cross attention as a PyTorch operator: gradients through views and broadcasts, torch.compile, opcheck; and the
example that runs the operators together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def autograd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transducer_loss_asr_gb300 import autograd as a

    return a


def _plain(q, k, v, k_lens, scale):
    G = q.shape[2] // k.shape[2]
    k, v = (t.repeat_interleave(G, 2).transpose(1, 2) for t in (k, v))
    s = q.transpose(1, 2) @ k.transpose(2, 3) * scale
    s = s.masked_fill((torch.arange(k.shape[2], device=k.device) >= k_lens[:, None])[:, None, None], -1e300)
    return (torch.softmax(s, 3) @ v).transpose(1, 2)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 4e-2)])
def test_gradients_through_views_and_broadcasts(autograd, dtype, tol):
    """k and v slices of one projection of frames that the batch shares: the gradient of the projection is
    what 64-bit autograd of the formula gives.  Tolerance: relative 2-norm, units of the type times ten."""
    g = torch.Generator(device="cuda").manual_seed(2)
    B, Lq, Lk, H, Hkv, D = 3, 37, 150, 4, 2, 64
    x = torch.randn(1, Lk, 2 * Hkv * D, generator=g, device="cuda")
    q0 = torch.randn(B, Lq, H, D, generator=g, device="cuda")
    go = torch.randn(B, Lq, H, D, generator=g, device="cuda")
    lens = torch.tensor([150, 77, 1], device="cuda")

    def run(f, dt):
        xs, qs = (t.to(dtype).to(dt).detach().clone().requires_grad_() for t in (x, q0))
        kv = xs.expand(B, -1, -1).unflatten(-1, (2, Hkv, D))
        out = f(qs, kv[:, :, 0], kv[:, :, 1])
        out.backward(go.to(dtype).to(dt))
        return out, xs.grad, qs.grad

    got = run(lambda q, k, v: autograd.cross_attention(q, k, v, lens), dtype)
    want = run(lambda q, k, v: _plain(q, k, v, lens, D ** -0.5), torch.float64)
    for a, b in zip(got, want):
        assert (a.double() - b).norm() <= tol * b.norm()


def test_module_compiled_and_opcheck(autograd):
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(2, 20, 4, 64, generator=g, device="cuda", dtype=torch.bfloat16).requires_grad_()
    k, v = (torch.randn(2, 90, 2, 64, generator=g, device="cuda", dtype=torch.bfloat16).requires_grad_() for _ in "kv")
    lens = torch.tensor([90, 33], device="cuda")
    m = autograd.CrossAttention()
    out = m(q, k, v, lens)
    grads = torch.autograd.grad(out.float().square().sum(), (q, k, v))
    compiled = torch.compile(m, fullgraph=True)
    out2 = compiled(q, k, v, lens)
    grads2 = torch.autograd.grad(out2.float().square().sum(), (q, k, v))
    assert torch.equal(out, out2)
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))
    torch.library.opcheck(torch.ops.tdt_gb300.cross_attention_forward.default,
                          (q.detach(), k.detach(), v.detach(), lens, None, None, 0.125),
                          test_utils=("test_schema", "test_faketensor"))


def test_the_example_runs_and_its_gradients_are_finite(autograd):
    spec = importlib.util.spec_from_file_location("attention_decoder", os.path.join(ROOT, "examples",
                                                                                   "attention_decoder.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    model, joint, tokens, score = mod.main(["--batch", "2", "--frames", "60", "--labels", "12", "--vocab", "300",
                                            "--width", "128", "--heads", "4", "--key-heads", "2", "--steps", "5"])
    assert tokens.shape == (2, 4, 5) and int(tokens.min()) >= 0 and int(tokens.max()) < 300
    assert bool(score.isfinite().all()) and bool((score <= 0).all())
    for p in list(model.parameters()) + [joint]:
        if p.grad is not None:
            assert bool(p.grad.isfinite().all())
    assert float(model.to_kv.weight.grad.abs().sum()) > 0
