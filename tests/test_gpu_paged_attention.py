"""Causal attention over a paged cache on the GPU against the formula in 64 bits.

Tolerances are bounds on what the kernels may round, worked out with the reference (see _reference): products and sums in float32
(unit 2^-24), exponentials good to 2^-20, and for the 16-bit types one rounding each of the weights and of the result (unit u).
Weights below 2^-31 of a row's largest may be lost (float16's least step).
"""
import math

import pytest
import torch

from paged_cases import E4M3, NAMES, TYPES, UNIT, i64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transducer_loss_asr_gb300 import binding as b

    return b


def _reference(q, k, v, kv_lens, q_lens, scale):
    """(out, its bound, lse, its bound) in 64 bits; q [B, Lq, H, D] of its type, k and v dense."""
    B, Lq, H, D = q.shape
    Lk, G, e32 = k.shape[1], H // k.shape[2], 2.0 ** -24
    u = UNIT[q.dtype]
    dev = q.device
    i = torch.arange(Lq, device=dev)
    real = i < q_lens[:, None]
    last = (kv_lens - q_lens)[:, None] + i
    seen = ((torch.arange(Lk, device=dev) <= last[..., None]) & real[..., None])[:, None]
    q = torch.where(real[..., None, None], q.double(), 0.0).transpose(1, 2)
    k, v = (t.transpose(1, 2).repeat_interleave(G, 1) for t in (k, v))
    s = torch.where(seen, q @ k.transpose(2, 3) * scale, -math.inf)
    lse = torch.logsumexp(s, 3)
    p = torch.where(seen, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    out = p @ v
    size = torch.where(seen, q.abs() @ k.abs().transpose(2, 3) * scale, 0.0)
    most = size.amax(3)
    ep = 2 * (D + 8 + Lk ** 0.5) * e32 * (most + 1.0) + 2.0 ** -20
    up, lost = (u, 2.0 ** -31) if q.dtype != torch.float32 else (0.0, 0.0)
    acc = (Lk + 8) ** 0.5 * 4 * e32
    tol = (p * (ep[..., None] + up + acc) + lost * seen) @ v.abs() + u * out.abs()
    t_lse = 2 * (D + 8) * e32 * (most + 1.0) + 2.0 ** -20 + 4 * e32 * torch.where(lse.isinf(), 0.0, lse.abs())
    tiny = 2.0 ** -24 if q.dtype == torch.float16 else 1e-30
    return out.transpose(1, 2), tol.transpose(1, 2) + tiny, lse, t_lse


def _near(name, x, value, bound, record=None, case=""):
    x = x.double()
    same = torch.equal(x.isinf(), value.isinf()) and torch.equal(x.isnan(), value.isnan())
    assert same, name
    fine = value.isfinite()
    if not fine.any():
        return
    ratio = ((x - value).abs()[fine] / bound[fine].clamp_min(1e-300)).max().item()
    if record:
        record(case, name, ratio, 1.0)
    assert ratio <= 1.0, "%s: error is %.3g of its bound" % (name, ratio)


def _queries(B, Lq, H, D, dtype, seed, q_lens, std=1.0, fused=True):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    q = (torch.randn(B, Lq, H + 2 if fused else H, D, generator=g, device="cuda") * std).to(dtype)[:, :, :H]
    for b, n in enumerate(q_lens):
        q[b, n:] = math.nan
    return q


def _check(binding, shape, dtype, cache_dtype, lens, q_lens=None, seed=0, scale=None, record=None, case="", q_std=1.0, fused=True,
           **how):
    """shape: (Lq, H, Hkv, D, page); lens: kv_lens; q_lens None: all Lq."""
    Lq, H, Hkv, D, page = shape
    B = len(lens)
    cache, table, k, v = make(binding, lens, Hkv, D, page, cache_dtype, seed, **how)
    counts = [Lq] * B if q_lens is None else q_lens
    q = _queries(B, Lq, H, D, dtype, seed, counts, q_std, fused)
    f = D ** -0.5 if scale is None else scale
    out, tol, lse, t_lse = _reference(q, k, v, i64(lens), i64(counts), f)
    ql = None if q_lens is None else i64(q_lens)
    got, got_lse = binding.tdt_paged_attn(q, cache, table, i64(lens), ql, scale=scale, need_lse=True)
    _near("out", got, out, tol, record, case)
    _near("lse", got_lse, lse, t_lse, record, case)
    alone, none = binding.tdt_paged_attn(q, cache, table, i64(lens), ql, scale=scale)
    assert none is None and torch.equal(alone, got)


SHAPES = [
    # Lq, H, Hkv, D, page, kv_lens
    (1, 1, 1, 8, 16, [1]),
    (1, 8, 8, 64, 16, [41, 1, 200]),
    (1, 8, 2, 128, 64, [333, 64, 65, 63]),
    (1, 16, 1, 64, 32, [500, 31]),
    (5, 6, 2, 80, 8, [130, 5, 9]),
    (41, 2, 2, 64, 16, [200, 41, 57]),
    (130, 3, 1, 40, 32, [130, 195]),
    (129, 2, 1, 128, 64, [257, 400]),
    (127, 4, 4, 96, 128, [383]),
    (300, 4, 1, 64, 256, [1000, 300]),
    (64, 4, 1, 128, 16, [2500]),
    (9, 2, 1, 5, 1, [70, 9]),
    (33, 2, 2, 250, 4, [70]),
]
CACHES = [(t, t) for t in TYPES] + [(t, E4M3) for t in TYPES]
IDS = ["%s-%s" % (NAMES[a], NAMES[b]) for a, b in CACHES]


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_whole(binding, record_margin, shape, dtype, cache_dtype):
    _check(binding, shape[:5], dtype, cache_dtype, shape[5], seed=1, record=record_margin,
           case="paged %s %s" % (NAMES[dtype], NAMES[cache_dtype]))


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("shape", [(1, 8, 2, 64, 16), (6, 4, 4, 128, 32), (70, 4, 2, 64, 8), (150, 2, 1, 96, 64)], ids=str)
def test_ragged(binding, record_margin, shape, dtype, cache_dtype):
    """Utterances without past, without new queries, without anything; a table wider than needed."""
    Lq = shape[0]
    _check(binding, shape, dtype, cache_dtype, [Lq, 300, 0, 129, max(1, Lq // 2), 128], [Lq, 0, 0, min(Lq, 5), max(1, Lq // 2), Lq if Lq < 128 else 7],
           seed=2, room=5, record=record_margin, case="paged ragged %s %s" % (NAMES[dtype], NAMES[cache_dtype]))


@pytest.mark.parametrize("dtype,cache_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, E4M3), (torch.float32, torch.float32)],
                         ids=["bf16", "f16-e4m3", "f32"])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("Lq", [1, 40])
def test_page_sizes(binding, page, Lq, dtype, cache_dtype):
    _check(binding, (Lq, 4, 2, 64, page), dtype, cache_dtype, [page + Lq, 3 * page + 77, Lq, 128 + Lq, 127 + Lq, 129 + Lq], seed=3)


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 3, 70])
def test_layouts_scale_and_large_scores(binding, dtype, cache_dtype, Lq):
    lens = [150, 97]
    for layout in ("heads", "fused"):
        if cache_dtype == E4M3 and layout == "fused":
            continue
        _check(binding, (Lq, 4, 2, 64, 16), dtype, cache_dtype, lens, seed=4, layout=layout, fused=False)
    _check(binding, (Lq, 4, 2, 64, 16), dtype, cache_dtype, lens, seed=5, scale=0.9)
    _check(binding, (Lq, 2, 2, 64, 32), dtype, cache_dtype, [400, 333], seed=6, std=6.0, q_std=6.0)  # one-hot softmax


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("Lq", [1, 4, 90])
@pytest.mark.parametrize("spread", [3.0, 12.0])
def test_quantised_rows_of_other_sizes(binding, dtype, Lq, spread):
    """Rows whose powers of two differ much, within a tile and between tiles."""
    std = 2.0 ** -10 if spread > 4 and dtype == torch.float16 else 1.0  # float16 results end at 65504
    _check(binding, (Lq, 4, 2, 128, 16), dtype, E4M3, [700, 300, 129], seed=7, spread=spread, std=std, scale=0.01)


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 2, 33])
def test_walks_of_every_length(binding, dtype, cache_dtype, Lq):
    for n in (1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385):
        if n >= Lq:
            _check(binding, (Lq, 2, 1, 64, 16), dtype, cache_dtype, [n, Lq], seed=8)


@pytest.mark.parametrize("dtype,cache_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, E4M3)], ids=["bf16", "bf16-e4m3"])
@pytest.mark.parametrize("Lq,H,Hkv,D", [(1, 8, 2, 128), (2, 4, 4, 64), (100, 4, 1, 128)])
def test_long_caches(binding, dtype, cache_dtype, Lq, H, Hkv, D):
    _check(binding, (Lq, H, Hkv, D, 64), dtype, cache_dtype, [9000, 5003, Lq], seed=9)


def test_rows_that_no_vector_load_fits(binding):
    g = torch.Generator(device="cuda").manual_seed(3)
    for dtype in TYPES:
        for Lq in (1, 20):
            base = torch.randn(10, 16, 3, 67, generator=g, device="cuda").to(dtype)
            q = torch.randn(2, Lq, 2, 67, generator=g, device="cuda").to(dtype)[..., 1:65]
            cache = binding.PagedCache(base[:, :, :1, 2:66], base[:, :, 1:2, 3:67])
            table = torch.tensor([[3, 1, 4, 5, 9], [2, 6, 0, 7, 8]], dtype=torch.int32, device="cuda")
            k, v = (t[table.long()].flatten(1, 2).double() for t in (cache.k, cache.v))
            lens, n = i64([80, 66]), i64([Lq, Lq])
            out, tol, lse, t_lse = _reference(q, k, v, lens, n, 0.125)
            wide = torch.full((2, Lq, 2, 67), 7.0, dtype=dtype, device="cuda")
            got, got_lse = binding.tdt_paged_attn(q, cache, table, lens, out=wide[..., 3:], need_lse=True)
            _near("out", got, out, tol)
            _near("lse", got_lse, lse, t_lse)
            assert bool((wide[..., :3] == 7.0).all())


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 6, 200])
def test_bad_lengths_and_pages(binding, dtype, cache_dtype, Lq):
    """Lengths that do not fit, and pages that are not there: NaN for that utterance, the others as they are."""
    cache, table, k, v = make(binding, [300] * 6, 2, 64, 16, cache_dtype, 5, poison=False)
    room = table.shape[1] * 16
    q = _queries(6, Lq, 4, 64, dtype, 5, [Lq] * 6)
    lens, counts = i64([room + 1, Lq - 1, -1, 300, 300, 300]), i64([Lq, Lq, Lq, Lq + 1, -1, Lq])
    out, lse = binding.tdt_paged_attn(q, cache, table, lens, counts, need_lse=True)
    assert bool(out[:5].isnan().all()) and bool(lse[:5].isnan().all())
    want, tol, _, _ = _reference(q, k, v, i64([300] * 6), i64([Lq] * 6), 0.125)
    _near("out", out[5], want[5], tol[5])
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 2], t[4, 0] = bad, bad
        out, lse = binding.tdt_paged_attn(q, cache, t, i64([300] * 6), need_lse=True)
        i = torch.arange(Lq, device="cuda") + 300 - Lq
        assert bool(out[1][i >= 32].isnan().all()) and bool(lse[1][:, i >= 32].isnan().all())
        assert bool(out[4].isnan().all()) and bool(lse[4].isnan().all())
        for b in (0, 2, 3, 5):
            _near("out", out[b], want[b], tol[b])


def test_hypotheses_that_share_pages(binding):
    """A beam: the pages of the common past are the same ones, each hypothesis has its own last page."""
    cache, table, k, v = make(binding, [100], 2, 64, 16, torch.bfloat16, 6, poison=False)
    beam = table[:, :7].expand(3, -1)  # stride 0: one table row for all
    q = _queries(3, 1, 4, 64, torch.bfloat16, 6, [1] * 3)
    lens = i64([100, 97, 64])
    out, tol, _, _ = _reference(q, k.expand(3, -1, -1, -1), v.expand(3, -1, -1, -1), lens, i64([1] * 3), 0.125)
    _near("out", binding.tdt_paged_attn(q, cache, beam, lens)[0], out, tol)


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 8, 140])
def test_same_inputs_same_bits_streams_graphs_and_given_workspace(binding, dtype, cache_dtype, Lq):
    cache, table, k, v = make(binding, [3000, Lq, 900], 2, 64, 32, cache_dtype, 7)
    q = _queries(3, Lq, 4, 64, dtype, 7, [Lq] * 3)
    lens = i64([3000, Lq, 900])
    want = binding.tdt_paged_attn(q, cache, table, lens, need_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = binding.tdt_paged_attn(q, cache, table, lens, need_lse=True)
    torch.cuda.current_stream().wait_stream(s)
    n = binding.tdt_paged_attn_workspace_size((3, Lq, 4, table.shape[1]), dtype, cache)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty(3, 4, Lq, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.tdt_paged_attn(q, cache, table, lens, out=out, lse=lse, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])


def test_a_graph_follows_lengths_and_tables(binding):
    """A captured decoding step: lengths, table and pages are read when it runs."""
    for dtype, cache_dtype in CACHES:
        cache, table, k, v = make(binding, [200, 150], 2, 64, 16, cache_dtype, 8)
        q = _queries(2, 1, 4, 64, dtype, 8, [1, 1])
        lens = i64([1, 1])
        out = torch.empty(2, 1, 4, 64, dtype=dtype, device="cuda")
        binding.tdt_paged_attn(q, cache, table, lens, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            binding.tdt_paged_attn(q, cache, table, lens, out=out)
        for n in ([200, 150], [17, 16], [128, 1]):
            lens.copy_(i64(n))
            graph.replay()
            want, tol, _, _ = _reference(q, k, v, i64(n), i64([1, 1]), 0.125)
            _near("out", out, want, tol)


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_offsets_past_32_bits(binding, cache_dtype):
    """Pages whose element offset does not fit 32 bits."""
    page, D = 256, 64
    n_pages = 2 ** 31 // (page * 2 * D) + 40
    pages = [torch.zeros(n_pages, page, 2, D, dtype=torch.uint8 if cache_dtype == E4M3 else cache_dtype, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, page, 2), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(2)
    table = torch.arange(n_pages - 4, n_pages, device="cuda").view(2, 2).to(torch.int32)
    dense = []
    for p in pages:
        x = torch.randn(4, page, 2, D, generator=g, device="cuda").to(cache_dtype)
        p[n_pages - 4:] = x.view(torch.uint8) if cache_dtype == E4M3 else x
        dense.append(x.double().view(2, 2 * page, 2, D))
    if cache_dtype == E4M3:
        cache = binding.PagedCache(*(p.view(E4M3) for p in pages), *scales)
    else:
        cache = binding.PagedCache(*pages)
    lens = i64([500, 257])
    for Lq in (1, 40):
        q = _queries(2, Lq, 4, D, torch.bfloat16, 1, [Lq] * 2)
        out, tol, _, _ = _reference(q, *dense, lens, i64([Lq] * 2), 0.125)
        _near("out", binding.tdt_paged_attn(q, cache, table, lens)[0], out, tol)


def test_nothing_to_do(binding):
    cache, table, _, _ = make(binding, [20], 2, 64, 16, torch.bfloat16)
    q = torch.empty(1, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert binding.tdt_paged_attn(q, cache, table, i64([20]))[0].shape == q.shape
    q = torch.full((1, 3, 4, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    out, lse = binding.tdt_paged_attn(q, cache, table[:, :0], i64([0]), i64([0]), need_lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 5, 20, 60, 130])
def test_queries_and_outputs_on_odd_addresses(binding, dtype, cache_dtype, Lq):
    """Pages that suit every kernel, queries and outputs that do not."""
    cache, table, k, v = make(binding, [300, Lq], 2, 64, 32, cache_dtype, 11)
    g = torch.Generator(device="cuda").manual_seed(Lq)
    q = torch.randn(2, Lq, 4, 67, generator=g, device="cuda").to(dtype)[..., 1:65]
    wide = torch.full((2, Lq, 4, 71), 7.0, dtype=dtype, device="cuda")
    lens = i64([300, Lq])
    out, tol, lse, t_lse = _reference(q, k, v, lens, i64([Lq, Lq]), 0.125)
    got, got_lse = binding.tdt_paged_attn(q, cache, table, lens, out=wide[..., 5:69], need_lse=True)
    _near("out", got, out, tol)
    _near("lse", got_lse, lse, t_lse)
    assert bool((wide[..., :5] == 7.0).all()) and bool((wide[..., 69:] == 7.0).all())


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 40])
def test_one_page_heads_of_stride_zero_and_shared_queries(binding, dtype, cache_dtype, Lq):
    cache, table, k, v = make(binding, [77, 50], 1, 64, 128, cache_dtype, 12)
    heads = [None if t is None else t.expand(-1, -1, 3, *([-1] * (t.dim() - 3))) for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    shared = binding.PagedCache(*heads)
    one = binding.PagedCache(*(None if t is None else t[int(table[0, 0]):int(table[0, 0]) + 1] for t in heads))
    g = torch.Generator(device="cuda").manual_seed(Lq)
    q = torch.randn(1, Lq, 6, 64, generator=g, device="cuda").to(dtype).expand(2, -1, -1, -1)
    k, v = (t.expand(-1, -1, 3, -1) for t in (k, v))
    lens = i64([77, 50])
    out, tol, _, _ = _reference(q, k, v, lens, i64([Lq, Lq]), 0.125)
    _near("out", binding.tdt_paged_attn(q, shared, table, lens)[0], out, tol)
    zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    _near("out", binding.tdt_paged_attn(q[:1], one, zero, lens[:1])[0], out[:1], tol[:1])


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("Lq", [3, 200])
def test_no_pages_and_no_new_rows(binding, dtype, cache_dtype, Lq):
    cache, table, _, _ = make(binding, [20], 2, 64, 16, cache_dtype)
    q = torch.full((2, Lq, 4, 64), math.nan, dtype=dtype, device="cuda")
    table = table.expand(2, -1)
    for t, lens in ((table[:, :0], [0, 0]), (table, [20, 0])):
        out, lse = binding.tdt_paged_attn(q, cache, t, i64(lens), i64([0, 0]), need_lse=True)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    out, _ = binding.tdt_paged_attn(q, cache, table[:, :0], i64([1, 0]), i64([1, 0]))
    assert bool(out[0].isnan().all()) and bool((out[1] == 0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("Lq", [1, 4, 40])
def test_value_rows_of_the_least_byte_come_first(binding, dtype, Lq):
    """Bytes that the caller set: value rows of byte 0 (2^-127) and, after every warp has had some, ordinary ones."""
    n, tiny = 2400, 1200
    cache, table, k, v = make(binding, [n, n - 300], 2, 64, 16, E4M3, 13)
    pages = table[:, :tiny // 16].long()
    cache.v_scales[pages] = 0
    v[:, :tiny] = cache.v[pages].double().flatten(1, 2) * 2.0 ** -127
    q = _queries(2, Lq, 4, 64, dtype, 13, [Lq] * 2)
    lens = i64([n, n - 300])
    out, tol, _, _ = _reference(q, k, v, lens, i64([Lq] * 2), 0.125)
    _near("out", binding.tdt_paged_attn(q, cache, table, lens)[0], out, tol)
