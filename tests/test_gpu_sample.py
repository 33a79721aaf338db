"""Drawing tokens on the GPU (tdt_sample) against the definition.

Where every weight is a power of two (T = log2(e), logits whole numbers) the draw is exact: whole-number arithmetic in Python
gives the same token.  Elsewhere the exponential is good to 2^-21, so the drawn token's stretch of the running sum has to
contain the target within 2^-20 of the weight that stays.
"""
import ctypes
import math
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

LOG2E = np.float32(1.4426950408889634)
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transducer_loss_asr_gb300 import binding as b

    return b


def _share(total, part24):
    return (int(total) * int(part24)) >> 24


def _kept(x, T, k, p, m):
    """(order of the tokens that stay, weights by token, those that top_p's cut may or may not include)."""
    with np.errstate(all="ignore"):
        x = x.astype(np.float32)
        X = np.nanmax(x)
        per = np.float32(0.0) if T == 0 else min(LOG2E / np.float32(T), np.float32(3.4e38))
        if np.isinf(X):
            z = np.where(x == X, 0.0, -100.0)
        else:
            z = np.maximum(((x - X).astype(np.float32) * per).astype(np.float32).astype(np.float64), -64.0)
        z = np.where(np.isnan(x), -64.0, z)
        w = np.rint(np.exp2(z) * 2.0 ** 31).astype(np.int64)
        order = np.argsort(-np.where(np.isnan(x), -np.inf, x), kind="stable")
    if T == 0:
        k = 1
    if 0 < k < len(x):
        order = order[:k]
    sure = len(order)
    p24 = int(np.rint(np.float32(p) * np.float32(2.0 ** 24)))
    if p24 < 1 << 24:
        run = np.cumsum(w[order])
        need = max(1, _share(run[-1], p24))
        before = run - w[order]
        slack = int(run[-1]) >> 19
        sure = max(1, int((before + slack < need).sum()))
        order = order[: max(1, int((before < need + slack).sum()))]
        exact = max(1, int((before < need).sum()))
    else:
        exact = len(order)
    floor = int(np.ceil(np.float32(m) * np.float32(2.0 ** 31)))
    stays = w[order] >= floor
    stays[0] = True
    cut = len(order) if stays.all() else int(np.argmin(stays))
    return order[:cut], w, min(sure, cut), min(exact, cut)


def _exact(x, u, T, k, p, m):
    order, w, _, n = _kept(x, T, k, p, m)
    ids = np.sort(order[:n])
    total = int(w[ids].sum())
    run = np.cumsum(w[ids])
    u24 = min(max(int(math.floor(np.float32(u) * np.float32(2.0 ** 24))), 0), (1 << 24) - 1)
    return int(ids[np.argmax(run > _share(total, u24))]), total


def _allowed(x, u, T, k, p, m, token):
    """Whether the token is the draw for weights within 2^-20 of the reference's."""
    order, w, sure, most = _kept(x, T, k, p, m)
    if token not in order:
        return False
    for n in {sure, most, len(order)}:
        ids = np.sort(order[:n])
        run = np.cumsum(w[ids])
        total, at = int(run[-1]), np.searchsorted(ids, token)
        if at < len(ids) and ids[at] == token:
            slack = total / 2.0 ** 20 + len(ids)
            if run[at] - w[token] - slack <= float(np.float32(u)) * total <= run[at] + slack:
                return True
    return False


def _settings(N, g, per_row, T, k, p, m):
    if not per_row:
        return dict(temperature=T, top_k=k, top_p=p, min_p=m), [(T, k, p, m)] * N
    f = torch.rand(4, N, generator=g, device="cuda")
    s = dict(temperature=T * (0.5 + f[0]), top_k=(f[1] * (2 * k + 1)).to(torch.int32),
             top_p=1.0 - (1.0 - p) * 2 * f[2] if p < 1 else torch.ones(N, device="cuda"), min_p=m * f[3])
    s["top_p"] = s["top_p"].clamp(0, 1).contiguous()
    rows = zip(*(s[n].cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p")))
    return s, [(t, int(kk), pp, mm) for t, kk, pp, mm in rows]


FILTERS = [(0, 1.0, 0.0), (1, 1.0, 0.0), (40, 1.0, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.1), (50, 0.95, 0.02), (5000, 0.5, 0.0),
           (0, 0.0, 0.0), (0, 0.999, 0.0), (300, 1.0, 1e-6), (0, 1.0, 1.0)]


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (64, 33), (40, 1000), (24, 8193), (6, 50257), (2, 140001)])
def test_whole_number_weights_are_exact(binding, dtype, N, V):
    """Weights are powers of two and ties are common: the token is the definition's, exactly."""
    g = torch.Generator(device="cuda").manual_seed(N * V)
    x = torch.randint(-24, 1, (N, V), generator=g, device="cuda").to(dtype)
    u = torch.rand(N, generator=g, device="cuda")
    xs = x.float().cpu().numpy()
    for k, p, m in FILTERS:
        tokens, logp = binding.tdt_sample(x, u, float(LOG2E), k, p, m)
        for i in range(N):
            want, total = _exact(xs[i], u[i].item(), float(LOG2E), k, p, m)
            assert tokens[i].item() == want, (k, p, m, i)
            z = float(xs[i][want] - xs[i].max())
            lp = (z - math.log2(total / 2.0 ** 31)) * math.log(2.0)
            assert abs(logp[i].item() - lp) <= 2e-6 * (1 + abs(lp))


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("N,V,width,std", [(7, 5, 5, 1.0), (200, 130, 133, 3.0), (50, 2048, 2051, 0.3),
                                           (30, 8193, 8198, 3.0), (30, 8193, 8193, 0.5), (4, 131072, 131075, 3.0)])
def test_random_logits(binding, dtype, per_row, N, V, width, std):
    g = torch.Generator(device="cuda").manual_seed(V + N)
    x = (torch.randn(N, width, generator=g, device="cuda") * std).to(dtype)[:, width - V:]
    u = torch.rand(N, generator=g, device="cuda")
    xs, us = x.float().cpu().numpy(), u.cpu().numpy()
    for k, p, m in FILTERS:
        for T in (0.7, 1.3):
            how, rows = _settings(N, g, per_row, T, k, p, m)
            tokens, logp = binding.tdt_sample(x, u, **how)
            tokens, logp = tokens.cpu().numpy(), logp.cpu().numpy()
            for i, (t, kk, pp, mm) in enumerate(rows):
                assert _allowed(xs[i], us[i], t, kk, pp, mm, tokens[i]), (T, k, p, m, i)
                assert logp[i] <= 1e-6 and logp[i] > -60


def test_greedy_and_ends_of_the_range(binding):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-3, 4, (20, 500), generator=g, device="cuda").float()
    first = x.argmax(1)  # ties: the lowest index, checked below
    for how in (dict(temperature=0.0), dict(top_k=1), dict(top_p=0.0), dict(temperature=1e-38), dict(temperature=1e-3, top_p=0.0)):
        if "temperature" in how and 0 < how["temperature"] < 1e-2 and "top_p" not in how:
            how = dict(how, top_k=1)
        tokens, logp = binding.tdt_sample(x, torch.rand(20, generator=g, device="cuda"), **how)
        want = [int(np.flatnonzero(r == r.max())[0]) for r in x.cpu().numpy()]
        assert tokens.tolist() == want and bool((logp == 0).all())
    assert first.shape == tokens.shape
    y = torch.zeros(3, 1000, device="cuda")  # equal weights: the token is floor(1000 u)
    tokens, logp = binding.tdt_sample(y, torch.tensor([0.0, 0.5, 1.0 - 2.0 ** -24], device="cuda"))
    assert tokens.tolist() == [0, 500, 999]
    assert torch.allclose(logp, torch.full((3,), -math.log(1000.0), device="cuda"), rtol=1e-6)
    tokens, _ = binding.tdt_sample(y, torch.tensor([-1.0, 1.0, math.nan], device="cuda"))
    assert tokens.tolist() == [0, 999, 0]


def test_infinite_and_missing_logits(binding):
    V = 3000
    x = torch.full((6, V), -math.inf, device="cuda")
    x[0, 17] = -5.0                       # one token left
    x[1, 40], x[1, 900] = math.inf, math.inf
    x[1, 41] = 3.0
    x[2] = math.nan                       # nothing to draw
    x[4, :] = math.nan
    x[4, 7], x[4, 2999] = 0.0, 0.0
    x[5, ::2] = torch.finfo(torch.float32).min
    x[5, 1] = 1.0
    u = torch.tensor([0.9, 0.6, 0.5, 0.5, 0.7, 0.99], device="cuda")
    for how in (dict(), dict(top_k=5), dict(top_p=0.999), dict(min_p=0.5), dict(temperature=0.3, top_k=2, top_p=0.99)):
        tokens, logp = binding.tdt_sample(x, u, **how)
        assert tokens.tolist() == [17, 900, -1, -1, 2999, 1], how
        assert logp[2:4].isnan().all() and torch.allclose(
            logp[[0, 1, 4, 5]], torch.tensor([0.0, -math.log(2.0), -math.log(2.0), 0.0], device="cuda"), atol=1e-6)
    tokens, logp = binding.tdt_sample(x, u, temperature=0.0)
    assert tokens.tolist() == [17, 40, -1, -1, 7, 1]


def test_bad_row_settings_touch_their_row_only(binding):
    x = torch.zeros(6, 100, device="cuda")
    x[:, 3] = 9.0
    u = torch.full((6,), 0.5, device="cuda")
    f = torch.float32
    t = torch.tensor([1.0, -1.0, math.nan, math.inf, 1.0, 1.0], device="cuda", dtype=f)
    k = torch.tensor([0, 0, 0, 0, -4, 7], device="cuda", dtype=torch.int32)
    tokens, logp = binding.tdt_sample(x, u, t, k)
    assert tokens.tolist() == [3, -1, -1, -1, -1, 3]
    p = torch.tensor([0.5, 1.1, -0.1, math.nan, 1.0, 0.0], device="cuda")
    tokens, _ = binding.tdt_sample(x, u, top_p=p)
    assert tokens.tolist() == [3, -1, -1, -1, 3, 3]
    tokens, _ = binding.tdt_sample(x, u, min_p=p)
    assert tokens.tolist() == [3, -1, -1, -1, 3, 3]


def test_frequencies_follow_the_probabilities(binding):
    """200,000 draws of one row: counts within five standard deviations of their expectation."""
    N, V = 200_000, 40
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(1, V, generator=g, device="cuda")
    tokens, _ = binding.tdt_sample(x.expand(N, V), torch.rand(N, generator=g, device="cuda"), 0.8, top_k=25)
    pr = torch.softmax(x[0].double() / 0.8, 0)
    keep = torch.zeros(V, dtype=torch.bool, device="cuda")
    keep[x[0].topk(25).indices] = True
    pr = torch.where(keep, pr, 0.0) / pr[keep].sum()
    counts = torch.bincount(tokens.long(), minlength=V).double()
    assert bool((counts[~keep] == 0).all())
    assert bool(((counts - N * pr).abs() <= 5 * (N * pr * (1 - pr)).sqrt() + 1)[keep].all())


def test_on_another_stream_and_in_a_graph(binding):
    g = torch.Generator(device="cuda").manual_seed(9)
    x, u = torch.randn(30, 8193, generator=g, device="cuda"), torch.rand(30, generator=g, device="cuda")
    want = binding.tdt_sample(x, u, 0.8, 50, 0.9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = binding.tdt_sample(x, u, 0.8, 50, 0.9)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = binding.tdt_sample(x, u, 0.8, 50, 0.9)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("V", [3000, 20000])
@pytest.mark.parametrize("X,temperatures", [(20.0, [3e-6 * 1.1 ** i for i in range(16)]), (1e8, [8.0 * 1.1 ** i for i in range(12)])])
def test_logits_on_a_coarse_grid(binding, V, X, temperatures):
    """Neighbouring floats that are far apart in units of the temperature: three tokens weigh anything, two of them equal
    and light; top-p takes one of the two, the one of lower index."""
    rows, ts, ps, want = [], [], [], []
    for T in temperatures:
        per = LOG2E / np.float32(T)
        x = np.float32(X)
        for _ in range(200):
            x = np.nextafter(x, np.float32(-np.inf))
            z = float(np.float32(np.float32(x - np.float32(X)) * per))
            if z < -15:
                break
            if z > -9:
                continue
            w = 2.0 ** (31 + z)  # the light ones' weight
            p24 = math.ceil((2.0 ** 31 + 0.5 * w) / (2.0 ** 31 + 2 * w) * 2.0 ** 24)
            if not 2.0 ** 31 + 0.2 * w < p24 / 2.0 ** 24 * (2.0 ** 31 + 2 * w) < 2.0 ** 31 + 0.8 * w:
                continue
            row = np.full(V, -np.inf, np.float32)
            row[1], row[1000], row[1001] = x, X, x
            rows.append(row)
            ts.append(T)
            ps.append(p24 / 2.0 ** 24)
    n = len(rows)
    assert n >= 20
    logits = torch.from_numpy(np.stack(rows)).cuda()
    how = dict(temperature=torch.tensor(ts, dtype=torch.float32, device="cuda"),
               top_p=torch.tensor(ps, dtype=torch.float32, device="cuda"))
    # the first of the kept tokens in the vocabulary's order, and the last
    for u, token in ((0.0, 1), (1.0 - 2.0 ** -24, 1000)):
        tokens, logp = binding.tdt_sample(logits, torch.full((n,), u, device="cuda"), **how)
        assert tokens.tolist() == [token] * n


HAMMER = r"""
#include <cstdint>
#include <atomic>
#include <thread>
#include <vector>
typedef int (*Sample)(const void *, const int64_t *, int64_t, int, const float *, const float *, const int32_t *,
                      const float *, const float *, double, int64_t, double, double, int32_t *, float *, void *);
// `threads` threads call at once, each with rows of its own length on a stream of its own; returns the calls that failed
extern "C" int hammer(Sample f, int threads, int times, void **logits, const int64_t *V, int64_t N, const float *u,
                      int32_t **tokens, float **logprobs, void **streams) {
  std::atomic<int> failed{0}, ready{0};
  std::vector<std::thread> all;
  for (int i = 0; i < threads; ++i)
    all.emplace_back([&, i] {
      const int64_t sizes[2] = {N, V[i]};
      for (++ready; ready < threads;) {
      }
      for (int k = 0; k < times; ++k)
        failed += f(logits[i], sizes, V[i], 0, u, nullptr, nullptr, nullptr, nullptr, 0.8, 50, 0.9, 0.0, tokens[i],
                    logprobs[i], streams[i]) != 0;
    });
  for (auto &t : all) t.join();
  return failed;
}
"""


@pytest.mark.parametrize("N,times", [(2, 3000), (400, 300)])
def test_threads_that_sample_rows_of_other_lengths(binding, tmp_path, N, times):
    """Host threads whose calls want other amounts of shared memory of one kernel do not make each other's launches fail."""
    (tmp_path / "hammer.cpp").write_text(HAMMER)
    so = str(tmp_path / "hammer.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-o", so, str(tmp_path / "hammer.cpp")],
                   check=True)
    g = torch.Generator(device="cuda").manual_seed(10)
    lengths = (1100, 16000, 1500, 12000)
    rows = [torch.randn(N, V, generator=g, device="cuda") for V in lengths]
    u = torch.rand(N, generator=g, device="cuda")
    want = [binding.tdt_sample(x, u, 0.8, 50, 0.9) for x in rows]
    got = [tuple(torch.empty_like(t) for t in pair) for pair in want]
    streams = [torch.cuda.Stream() for _ in rows]
    torch.cuda.synchronize()
    n = len(rows)

    def addresses(x):
        return (ctypes.c_void_p * n)(*x)

    failed = ctypes.CDLL(so).hammer(
        ctypes.cast(binding.lib.tdt_sample, ctypes.c_void_p), n, times, addresses(x.data_ptr() for x in rows),
        (ctypes.c_int64 * n)(*lengths), ctypes.c_int64(N), ctypes.c_void_p(u.data_ptr()),
        addresses(t.data_ptr() for t, _ in got), addresses(l.data_ptr() for _, l in got),
        addresses(s.cuda_stream for s in streams))
    torch.cuda.synchronize()
    assert failed == 0
    for (t, l), (t2, l2) in zip(want, got):
        assert torch.equal(t, t2) and torch.equal(l, l2)


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V,std", [(50, 130, 3.0), (30, 2048, 0.3), (20, 8193, 3.0), (4, 131072, 3.0)])
def test_log_probabilities(binding, dtype, N, V, std):
    """log-probability of the drawn token among those that stay, in 64 bits from the definition's weights.

    Bound: weights good to 2^-20 and one unit each (the exponential's error may move the last rounding), float32
    arithmetic on numbers of the size of z and of the logarithm; top-p's cut may fall one token to either side."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(N, V, generator=g, device="cuda") * std).to(dtype)
    u = torch.rand(N, generator=g, device="cuda")
    xs = x.float().cpu().numpy()
    for k, p, m in FILTERS:
        for T in (0.7, 1.3):
            tokens, logp = (t.cpu().numpy() for t in binding.tdt_sample(x, u, T, k, p, m))
            for i in range(N):
                order, w, sure, most = _kept(xs[i], T, k, p, m)
                z = float(np.float32(np.float32(xs[i][tokens[i]] - xs[i].max()) * (LOG2E / np.float32(T))))
                off = math.inf
                for n in range(sure, len(order) + 1):
                    total = int(w[order[:n]].sum())
                    lg = math.log2(total / 2.0 ** 31)
                    bound = (2.0 ** -20 + n / total + 2.0 ** -22 * (1 + abs(z) + abs(lg))) * math.log(2.0) * 2
                    off = min(off, abs(logp[i] - (z - lg) * math.log(2.0)) / bound)
                    if off <= 1:
                        break
                assert off <= 1, (T, k, p, m, i, off)
