"""Writing label states into pages and reading them back, on the GPU: exact, by the definition in 64 bits (paged_cases.quantised)."""
import math

import pytest
import torch

from paged_cases import E4M3, NAMES, TYPES, i64, quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transducer_loss_asr_gb300 import binding as b

    return b


def _new(binding, n_pages, page, Hkv, D, dtype, byte=0x5a):
    """A cache of bytes `byte`: what no row goes to has to keep them."""
    c = binding.PagedCache.empty(n_pages, page, Hkv, D, dtype)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            t.view(torch.uint8).fill_(byte)
    return c


def _rows(g, B, L, Hkv, D, dtype, spread=8.0):
    x = torch.randn(B, L, 2 * Hkv + 1, D, generator=g, device="cuda") * torch.exp2(
        (torch.rand(B, L, 2 * Hkv + 1, 1, generator=g, device="cuda") * 2 - 1) * spread)
    return x.to(dtype)


CACHES = [(t, t) for t in TYPES] + [(t, E4M3) for t in TYPES]
IDS = ["%s-%s" % (NAMES[a], NAMES[b]) for a, b in CACHES]


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
@pytest.mark.parametrize("B,L,Hkv,D,page", [(1, 1, 1, 1, 1), (3, 1, 8, 64, 16), (4, 41, 2, 128, 32), (2, 7, 3, 40, 8), (2, 300, 1, 96, 64),
                                            (2, 5, 2, 5, 4), (1, 9, 2, 250, 2), (2, 33, 4, 256, 128)])
def test_write_and_read_back(binding, B, L, Hkv, D, page, dtype, cache_dtype):
    g = torch.Generator(device="cuda").manual_seed(B * L * D)
    x = _rows(g, B, L, Hkv, D, dtype)
    k, v = x[:, :, :Hkv], x[:, :, Hkv:2 * Hkv]
    past = torch.randint(0, 3 * page + 1, (B,), generator=g, device="cuda")
    counts = torch.randint(0, L + 1, (B,), generator=g, device="cuda")
    counts[0] = L
    lens = past + counts
    M = (3 * page + L + page - 1) // page
    cache = _new(binding, B * M + 2, page, Hkv, D, cache_dtype)
    table = torch.randperm(B * M + 2, generator=g, device="cuda")[:B * M].view(B, M).to(torch.int32)
    for b in range(B):
        k[b, counts[b]:], v[b, counts[b]:] = math.nan, math.inf  # not read
    binding.tdt_cache_write(k, v, cache, table, lens, counts)
    touched = torch.zeros(B * M + 2, page, dtype=torch.bool, device="cuda")
    for pages, scales, src in ((cache.k, cache.k_scales, k), (cache.v, cache.v_scales, v)):
        for b in range(B):
            n = int(counts[b])
            pos = int(past[b]) + torch.arange(n, device="cuda")
            at = (table[b].long()[pos // page], pos % page)
            touched[at] = True
            if cache_dtype == E4M3:
                value, byte = quantised(src[b, :n])
                assert torch.equal(scales[at], byte)
                assert torch.equal(pages[at].double() * torch.exp2(byte.double() - 127)[..., None], value)
            else:
                assert torch.equal(pages[at], src[b, :n])
        assert bool((pages.contiguous().view(torch.uint8).view(B * M + 2, page, -1)[~touched] == 0x5a).all())
        if scales is not None:
            assert bool((scales[~touched] == 0x5a).all())
    for out_dtype in TYPES:
        got = binding.tdt_cache_read(cache, table, lens, counts, L, out_dtype)
        for y, src in zip(got, (k, v)):
            for b in range(B):
                n = int(counts[b])
                value = quantised(src[b, :n])[0] if cache_dtype == E4M3 else src[b, :n].double()
                assert torch.equal(y[b, :n], value.to(out_dtype)), (out_dtype, b)
                assert bool((y[b, n:] == 0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
def test_every_value_of_a_type_and_ties(binding, dtype):
    """All 16-bit patterns (random ones of float32) as elements of rows whose largest element fixes the power of two: steps, ties and
    what lies below the least step come out as the definition says."""
    if dtype == torch.float32:
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randint(-2 ** 31, 2 ** 31, (2 ** 16,), generator=g, device="cuda").to(torch.int32).view(torch.float32)
    else:
        x = torch.arange(-2 ** 15, 2 ** 15, device="cuda").to(torch.int16).view(dtype)
    x = torch.where(x.isfinite(), x, 0.0).view(1, -1, 1, 16).clone()
    exact = (torch.arange(-512, 512, device="cuda") / 32.0).repeat(16).view(1, -1, 1, 16)  # ties of steps of 1/4 up to 2
    top = torch.tensor([448.0, 1.75, 1.7578125, 3.5, 256.0, 0.9375], device="cuda")
    for extra in [None] + top.tolist():
        for src in (x, exact.to(dtype)):
            src = src.clone()
            if extra is not None:
                src = torch.where(src.float().abs() <= extra, src, 0.0)
                src[..., 0] = extra
            L = src.shape[1]
            cache = _new(binding, L // 256 + 1, 256, 1, 16, E4M3)
            table = torch.arange(L // 256 + 1, device="cuda").to(torch.int32)[None]
            binding.tdt_cache_write(src, -src, cache, table, i64([L]))
            k, v = binding.tdt_cache_read(cache, table, i64([L]), None, L, torch.float32)
            value, byte = quantised(src)
            assert torch.equal(k.double(), value.to(torch.float32).double()) and torch.equal(v, -k)
            assert torch.equal(cache.k_scales.view(-1)[:L], byte.view(-1))


@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
def test_rows_that_are_not_finite_or_all_zero(binding, dtype):
    x = torch.randn(1, 6, 1, 64, device="cuda").to(dtype)
    x[0, 1, 0, 63], x[0, 2, 0, 0], x[0, 3, 0, 7], x[0, 4] = math.nan, math.inf, -math.inf, 0.0
    cache = _new(binding, 1, 8, 1, 64, E4M3)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    binding.tdt_cache_write(x, x, cache, table, i64([6]))
    k, _ = binding.tdt_cache_read(cache, table, i64([6]), None, 6, dtype)
    assert cache.k_scales[0, 1:4, 0].tolist() == [255] * 3 and bool(k[0, 1:4].isnan().all())
    assert bool((k[0, 4] == 0).all()) and bool(k[0, [0, 5]].isfinite().all())
    # pages of their own type keep them
    cache = _new(binding, 1, 8, 1, 64, dtype)
    binding.tdt_cache_write(x, x, cache, table, i64([6]))
    k, _ = binding.tdt_cache_read(cache, table, i64([6]), None, 6, dtype)
    assert torch.equal(k.nan_to_num(7.0), x.nan_to_num(7.0)) and torch.equal(k.isnan(), x.isnan())


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_bad_lengths_and_pages(binding, cache_dtype):
    """Nothing is written for them, and they read as NaN."""
    page, L = 16, 10
    cache = _new(binding, 8, page, 2, 64, cache_dtype)
    table = torch.arange(8, device="cuda").view(4, 2).to(torch.int32)
    x = torch.randn(4, L, 2, 64, device="cuda").to(torch.bfloat16)
    for lens, counts in (([33, 9, -1, 20], [10, 10, 10, 11]), ([20, 20, 20, 20], [-1, 11, 100, -2 ** 40]), ([2 ** 40] * 4, [10] * 4)):
        binding.tdt_cache_write(x, x, cache, table, i64(lens), i64(counts))
        for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
            assert t is None or bool((t.view(torch.uint8) == 0x5a).all())
        k, v = binding.tdt_cache_read(cache, table, i64(lens), i64(counts), L, torch.bfloat16)
        assert bool(k.isnan().all()) and bool(v.isnan().all())
    for bad in (-1, 8, 2 ** 31 - 1):
        t = table.clone()
        t[:, 1] = bad
        binding.tdt_cache_write(x, x, cache, t, i64([20] * 4))
        k, _ = binding.tdt_cache_read(cache, t, i64([20] * 4), None, L, torch.bfloat16)
        assert bool(k[:, 6:].isnan().all()) and bool(k[:, :6].isfinite().all())
        untouched = cache.k.view(torch.uint8)[1::2]
        assert bool((untouched == 0x5a).all())


@pytest.mark.parametrize("dtype,cache_dtype", CACHES, ids=IDS)
def test_layouts_offsets_and_given_outputs(binding, dtype, cache_dtype):
    """Heads before places, rows on odd addresses, inputs shared by the batch, outputs in slices."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(1, 20, 2, 67, generator=g, device="cuda").to(dtype).expand(2, -1, -1, -1)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    for D, off in ((64, 0), (64, 1), (61, 3)):
        k, v = x[..., off:off + D], x[..., :D]
        base = [torch.zeros(4, 2, 16, D + 3, dtype=cache_dtype, device="cuda").transpose(1, 2)[..., 3:] for _ in range(2)]
        scales = [torch.zeros(4, 2, 16, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)] if cache_dtype == E4M3 else []
        cache = binding.PagedCache(*base, *scales)
        binding.tdt_cache_write(k, v, cache, table, i64([30, 21]))
        wide = torch.full((2, 20, 2, 2, D + 1), 7.0, dtype=dtype, device="cuda")
        got = binding.tdt_cache_read(cache, table, i64([30, 21]), None, 20, dtype, k=wide[:, :, 0, :, 1:], v=wide[:, :, 1, :, 1:])
        for y, src in zip(got, (k, v)):
            want = quantised(src)[0].to(dtype) if cache_dtype == E4M3 else src
            assert torch.equal(y, want)
        assert bool((wide[..., 0] == 7.0).all())


def test_offsets_past_32_bits(binding):
    page, D = 256, 128
    n_pages = 2 ** 31 // (page * D) + 6
    for cache_dtype in (torch.bfloat16, E4M3):
        cache = binding.PagedCache.empty(n_pages, page, 1, D, cache_dtype)
        x = torch.randn(1, 300, 1, D, device="cuda").to(torch.bfloat16)
        table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device="cuda")
        binding.tdt_cache_write(x, -x, cache, table, i64([400]))
        k, v = binding.tdt_cache_read(cache, table, i64([400]), None, 300, torch.bfloat16)
        want = quantised(x)[0].to(x.dtype) if cache_dtype == E4M3 else x
        assert torch.equal(k, want) and torch.equal(v, -want)
        del cache


def test_in_a_graph_and_on_another_stream(binding):
    cache = _new(binding, 8, 16, 2, 64, E4M3)
    table = torch.arange(8, device="cuda").view(2, 4).to(torch.int32)
    x = torch.randn(2, 1, 2, 64, device="cuda").to(torch.bfloat16)
    lens = i64([1, 1])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        binding.tdt_cache_write(x, x, cache, table, lens)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        binding.tdt_cache_write(x, x, cache, table, lens)
    rows = []
    for n in range(1, 40):  # a decoding loop: the replayed write follows the lengths and the rows
        lens.fill_(n)
        x.copy_(torch.randn(2, 1, 2, 64, device="cuda"))
        rows.append(x.clone())
        graph.replay()
    k, _ = binding.tdt_cache_read(cache, table, i64([39, 39]), None, 39, torch.bfloat16)
    assert torch.equal(k, quantised(torch.cat(rows, 1))[0].to(torch.bfloat16))
