"""The paged cache, its attention and token log-probabilities refuse bad arguments on the host, before touching any device (no GPU
here: only calls that fail validation, or have nothing to do, are made)."""
import ctypes
import struct

import pytest
import torch

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from transducer_loss_asr_gb300 import build

    build.build()
    from transducer_loss_asr_gb300 import binding

    return binding


def _arr(x):
    return None if x is None else (ctypes.c_int64 * len(x))(*x)


def _cache(k=FAKE, v=FAKE, ks=None, vs=None, n_pages=10, page_size=16, heads=2, dim=64, strides=None, dtype=2):
    if dtype == 3 and ks is None:
        ks = vs = FAKE
    one = [page_size * heads * dim, heads * dim, dim]
    s = [page_size * heads, heads, 1] if dtype == 3 else [0, 0, 0]
    strides = one + one + s + s if strides is None else strides
    return struct.pack("=4Q4q12qi4x", k or 0, v or 0, ks or 0, vs or 0, n_pages, page_size, heads, dim, *strides, dtype)


def test_the_bindings_struct_is_the_headers(lib):
    assert len(_cache()) == struct.calcsize("@4P4q12qi") + 4  # padded to its alignment


ROWS = dict(k=FAKE, v=FAKE, sizes=[2, 5, 3], strides=[640, 128, 64, 640, 128, 64], dtype=2, cache={}, table=FAKE, table_stride=3,
            kv_lens=FAKE, q_lens=FAKE)


def _rows(lib, read, over):
    a = dict(ROWS, **over)
    cache = None if a["cache"] is None else _cache(**a["cache"])
    if read:
        return lib.lib.tdt_cache_read(cache, a["table"], a["table_stride"], a["kv_lens"], a["q_lens"], _arr(a["sizes"]), _arr(a["strides"]),
                                      a["dtype"], a["k"], a["v"], None)
    return lib.lib.tdt_cache_write(a["k"], a["v"], _arr(a["sizes"]), _arr(a["strides"]), a["dtype"], cache, a["table"], a["table_stride"],
                                   a["kv_lens"], a["q_lens"], None)


CACHE_FAULTS = [
    (dict(cache=None), -1),
    (dict(cache=dict(k=None)), -1),
    (dict(cache=dict(v=None)), -1),
    (dict(cache=dict(dtype=3, ks=FAKE, vs=None)), -1),
    (dict(cache=dict(dtype=4)), -4),
    (dict(cache=dict(dtype=-1)), -4),
    (dict(cache=dict(k=FAKE + 1)), -11),
    (dict(cache=dict(heads=0)), -14),
    (dict(cache=dict(dim=0)), -14),
    (dict(cache=dict(dim=257)), -14),
    (dict(cache=dict(n_pages=0)), -17),
    (dict(cache=dict(n_pages=1 << 31)), -17),
    (dict(cache=dict(page_size=0)), -17),
    (dict(cache=dict(page_size=24)), -17),
    (dict(cache=dict(page_size=1 << 17)), -17),
    (dict(cache=dict(strides=[-2048, 128, 64] + [2048, 128, 64] + [0] * 6)), -3),
    (dict(table=None), -1),
    (dict(kv_lens=None), -1),
    (dict(table=FAKE + 2), -11),
    (dict(kv_lens=FAKE + 4), -11),
    (dict(q_lens=FAKE + 4), -11),
    (dict(table_stride=-1), -3),
]


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("over,code", CACHE_FAULTS + [
    (dict(sizes=None), -1),
    (dict(strides=None), -1),
    (dict(k=None), -1),
    (dict(v=None), -1),
    (dict(k=FAKE + 1), -11),
    (dict(dtype=3), -4),
    (dict(strides=[640, 128, -64, 640, 128, 64]), -3),
    (dict(sizes=[-1, 5, 3]), -2),
    (dict(sizes=[2, -5, 3]), -2),
    (dict(sizes=[1 << 20, 1 << 20, 3]), -2),
    (dict(sizes=[2, 5, -3]), -17),
    (dict(sizes=[2, 5, 1 << 26]), -17),
    (dict(sizes=[0, 5, 3], k=None, table=None), 0),
    (dict(sizes=[2, 0, 3], k=None, table=None), 0),
])
def test_cache_rows_are_refused(lib, read, over, code):
    assert _rows(lib, read, over) == code


def test_cache_writes_and_reads_that_overlap_themselves(lib):
    assert _rows(lib, False, dict(cache=dict(strides=[2048, 0, 64] + [2048, 128, 64] + [0] * 6))) == -3      # places share addresses
    assert _rows(lib, False, dict(cache=dict(strides=[2048, 128, 64] + [2048, 128, 32] + [0] * 6))) == -3
    assert _rows(lib, False, dict(cache=dict(dtype=3, strides=[2048, 128, 64] * 2 + [32, 2, 1] + [32, 0, 1]))) == -3
    assert _rows(lib, True, dict(strides=[640, 128, 64, 640, 0, 64])) == -3
    assert _rows(lib, False, dict(dtype=0)) == -4       # float32 rows, bfloat16 pages


ATTN = dict(q=FAKE, sizes=[2, 5, 4, 3], strides=[1280, 256, 64, 1280, 256, 64], dtype=2, cache={}, table=FAKE, table_stride=3,
            kv_lens=FAKE, q_lens=FAKE, scale=0.125, out=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 40)


def _attn(lib, over):
    a = dict(ATTN, **over)
    cache = None if a["cache"] is None else _cache(**a["cache"])
    return lib.lib.tdt_paged_attn(a["q"], _arr(a["sizes"]), _arr(a["strides"]), a["dtype"], cache, a["table"], a["table_stride"],
                                  a["kv_lens"], a["q_lens"], a["scale"], a["out"], a["lse"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("over,code", CACHE_FAULTS + [
    (dict(sizes=None), -1),
    (dict(strides=None), -1),
    (dict(q=None), -1),
    (dict(out=None), -1),
    (dict(q=FAKE + 1), -11),
    (dict(out=FAKE + 1), -11),
    (dict(lse=FAKE + 2), -11),
    (dict(dtype=3), -4),
    (dict(dtype=1), -4),                                # float16 queries, bfloat16 pages
    (dict(sizes=[2, 5, 3, 3]), -14),
    (dict(sizes=[2, 5, 0, 3]), -14),
    (dict(sizes=[-2, 5, 4, 3]), -2),
    (dict(sizes=[2, 1 << 30, 4, 3]), -2),
    (dict(sizes=[1 << 20, 1 << 20, 4, 3]), -2),
    (dict(sizes=[2, 5, 4, 1 << 26]), -17),
    (dict(sizes=[2, 5, 4, -1]), -17),
    (dict(strides=[1280, 256, 64, 1280, 256, 32]), -3),  # heads of out overlap
    (dict(strides=[-1280, 256, 64, 1280, 256, 64]), -3),
    (dict(scale=0.0), -15),
    (dict(scale=float("nan")), -15),
    (dict(scale=float("inf")), -15),
    (dict(sizes=[0, 5, 4, 3], q=None), 0),
    (dict(sizes=[2, 0, 4, 3], q=None), 0),
])
def test_paged_attention_refuses(lib, over, code):
    assert _attn(lib, over) == code


def test_paged_attention_workspace(lib):
    """Sizes that need scratch refuse too little of it; invalid ones need none."""
    for cache, dtype in ((dict(), 2), (dict(dtype=3), 2), (dict(dtype=0), 0), (dict(dtype=3, dim=128), 1)):
        for sizes in ([1, 1, 4, 200], [1, 100, 4, 200], [4, 500, 4, 2000]):
            need = lib.lib.tdt_paged_attn_workspace_size(_arr(sizes), dtype, _cache(**cache))
            if need:
                a = dict(sizes=sizes, cache=cache, dtype=dtype, table_stride=sizes[3])
                assert _attn(lib, dict(a, nbytes=need - 1)) == -9
                assert _attn(lib, dict(a, ws=None)) == -1
                assert _attn(lib, dict(a, ws=FAKE + 8)) == -11
    assert lib.lib.tdt_paged_attn_workspace_size(_arr([2, 5, 3, 3]), 2, _cache()) == 0
    assert lib.lib.tdt_paged_attn_workspace_size(_arr([2, 5, 4, 3]), 2, None) == 0


LOGP = dict(logits=FAKE, sizes=[3, 50, 4], strides=[50, 50], dtype=0, tokens=FAKE, entropy=FAKE, stats=FAKE, top=FAKE, a=FAKE, b=FAKE, c=FAKE,
            grad=FAKE + (1 << 20), logprobs=FAKE, top_lp=FAKE)


def _logp(lib, which, over):
    x = dict(LOGP, **over)
    sizes, strides = _arr(x["sizes"]), _arr(x["strides"])
    if which == "fwd":
        return lib.lib.tdt_token_logprobs_fwd(x["logits"], sizes, x["strides"][0], x["dtype"], x["tokens"], x["logprobs"], x["entropy"],
                                              x["stats"], x["top"], x["top_lp"], None)
    if which == "bwd":
        return lib.lib.tdt_token_logprobs_bwd(x["logits"], sizes, strides, x["dtype"], x["tokens"], x["entropy"], x["stats"], x["top"],
                                              x["a"], x["b"], x["c"], x["grad"], None)
    return lib.lib.tdt_token_logprobs_fwd_bwd(x["logits"], sizes, strides, x["dtype"], x["tokens"], x["a"], x["b"], x["logprobs"],
                                              x["entropy"], x["stats"], x["top"], x["top_lp"], x["grad"], None)


ALL, FWD, BWD = ("fwd", "bwd", "both"), ("fwd", "both"), ("bwd", "both")


@pytest.mark.parametrize("where,over,code", [
    (ALL, dict(sizes=None), -1),
    (ALL, dict(logits=None), -1),
    (ALL, dict(tokens=None), -1),
    (ALL, dict(sizes=[-1, 50, 4]), -2),
    (ALL, dict(sizes=[3, 0, 0]), -2),
    (ALL, dict(sizes=[3, (1 << 24) + 1, 4]), -2),
    (ALL, dict(sizes=[3, 50, -1]), -18),
    (ALL, dict(sizes=[3, 50, 51]), -18),
    (ALL, dict(sizes=[3, 5000, 65]), -18),
    (ALL, dict(strides=[-50, 50]), -3),
    (ALL, dict(dtype=3), -4),
    (ALL, dict(logits=FAKE + 2), -11),
    (ALL, dict(tokens=FAKE + 4), -11),
    (ALL, dict(stats=FAKE + 4), -11),
    (ALL, dict(entropy=FAKE + 2), -11),
    (FWD, dict(logprobs=None), -1),
    (FWD, dict(top=None), -1),
    (FWD, dict(top_lp=None), -1),
    (FWD, dict(logprobs=FAKE + 2), -11),
    (BWD, dict(grad=None), -1),
    (BWD, dict(grad=FAKE + (1 << 20) + 2), -11),
    (BWD, dict(strides=[50, 49]), -3),
    (BWD, dict(strides=[50, 0]), -3),
    (BWD, dict(grad=FAKE + 4), -13),
    (BWD, dict(grad=FAKE, strides=[50, 60]), -13),
    (BWD, dict(a=FAKE + 2), -11),
    (("bwd",), dict(stats=None), -1),
    (("bwd",), dict(entropy=None), -1),
    (("bwd",), dict(top=None), -1),
    (ALL, dict(sizes=[0, 50, 4], logits=None), 0),
])
def test_token_logprobs_refuse(lib, where, over, code):
    for which in where:
        if over.get("sizes", 0) is None and which == "fwd":
            assert lib.lib.tdt_token_logprobs_fwd(FAKE, None, 50, 0, FAKE, FAKE, None, None, None, None, None) == code
        else:
            assert _logp(lib, which, over) == code, which


def test_new_status_texts(lib):
    for code in (-17, -18):
        assert lib.tdt_status_string(code) != "unknown status"


def test_binding_refuses_bad_caches(lib):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.PagedCache(k[0], k[0])
    with pytest.raises(ValueError):
        lib.PagedCache(k, k[:, :8])
    with pytest.raises(TypeError):
        lib.PagedCache(k.double(), k.double())
    with pytest.raises(ValueError):
        lib.PagedCache(k, k.float())
    with pytest.raises(ValueError):
        lib.PagedCache(k.transpose(2, 3), k.transpose(2, 3))
    with pytest.raises(ValueError):
        lib.PagedCache(k, k, torch.zeros(4, 16, 2, dtype=torch.uint8), torch.zeros(4, 16, 2, dtype=torch.uint8))
    q = k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        lib.PagedCache(q, q)
    with pytest.raises(ValueError):
        lib.PagedCache(q, q, torch.zeros(4, 16, 2), torch.zeros(4, 16, 2))
    c = lib.PagedCache.empty(4, 16, 2, 64, torch.float8_e4m3fn, device="cpu")
    assert c.k.shape == (4, 16, 2, 64) and c.v_scales.shape == (4, 16, 2)


def test_binding_refuses_bad_cache_calls(lib):
    cache = lib.PagedCache.empty(4, 16, 2, 64, torch.bfloat16, device="cpu")
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    x = torch.zeros(3, 5, 2, 64, dtype=torch.bfloat16)
    for bad in (dict(k=x[0]), dict(v=x[:, :4]), dict(k=x[..., :32], v=x[..., :32]), dict(k=x[:, :, :1], v=x[:, :, :1]), dict(page_table=table.long()),
                dict(page_table=table[:2]), dict(page_table=torch.zeros(2, 3, dtype=torch.int32).t()), dict(kv_lens=lens.int()),
                dict(kv_lens=lens[:2]), dict(q_lens=lens.int()), {}):  # the last: a CPU tensor
        a = dict(dict(k=x, v=x, cache=cache, page_table=table, kv_lens=lens, q_lens=lens), **bad)
        with pytest.raises(ValueError):
            lib.tdt_cache_write(**a)
    for bad in (dict(k=x.double(), v=x.double()), dict(v=x.float()), dict(k=x.float(), v=x.float())):
        with pytest.raises(TypeError):
            lib.tdt_cache_write(**dict(dict(k=x, v=x, cache=cache, page_table=table, kv_lens=lens), **bad))
    with pytest.raises(TypeError):
        lib.tdt_cache_read(cache, table, lens, None, 5, torch.float64)
    with pytest.raises(ValueError):
        lib.tdt_cache_read(cache, table, lens, None, 5, torch.float32, k=torch.zeros(3, 4, 2, 64))
    with pytest.raises(ValueError):
        lib.tdt_cache_read(cache, table, lens, None, 5, torch.float32)
    q = torch.zeros(3, 5, 4, 64, dtype=torch.bfloat16)
    for bad in (dict(q=q[0]), dict(q=q[..., :32]), dict(page_table=table[:1]), dict(kv_lens=lens.int()), dict(out=q[:, :4]),
                dict(lse=torch.zeros(3, 5, 4)), dict(workspace=torch.zeros(8)), {}):
        with pytest.raises(ValueError):
            lib.tdt_paged_attn(**dict(dict(q=q, cache=cache, page_table=table, kv_lens=lens), **bad))
    for bad in (q.double(), q.float()):
        with pytest.raises(TypeError):
            lib.tdt_paged_attn(bad, cache, table, lens)


def test_binding_refuses_bad_scored_rows(lib):
    x, t, w = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    with pytest.raises(ValueError):
        lib.tdt_token_logprobs_fwd(x[0], t)
    with pytest.raises(TypeError):
        lib.tdt_token_logprobs_fwd(x.double(), t)
    for bad in (t.int(), t[:2], torch.zeros(6, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError):
            lib.tdt_token_logprobs_fwd(x, bad)
    r = lib.TokenLogprobs(w, w, torch.zeros(3, 2), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4))
    for bad in (dict(grad_logprobs=w[:2]), dict(grad_entropy=w.double()), dict(grad_top=torch.zeros(3, 5)), dict(grad_out=x[:, :4]),
                dict(result=r._replace(stats=torch.zeros(3))), dict(result=r._replace(top_tokens=None), grad_top=torch.zeros(3, 4)), {}):
        with pytest.raises(ValueError):
            lib.tdt_token_logprobs_bwd(**dict(dict(logits=x, tokens=t, result=r, grad_logprobs=w), **bad))
    with pytest.raises(ValueError):
        lib.tdt_token_logprobs_fwd_bwd(x, t, w, grad_out=torch.zeros(50, 3).t())


def test_token_logprobs_op_fake_shapes_and_cpu_rejection(lib):
    from transducer_loss_asr_gb300 import autograd

    x, t = torch.empty(6, 50, device="meta"), torch.empty(6, dtype=torch.int64, device="meta")
    lp, ent, stats, top, top_lp = torch.ops.tdt_gb300.token_logprobs_forward(x, t, 4)
    assert lp.shape == ent.shape == (6,) and stats.shape == (6, 2) and top.shape == top_lp.shape == (6, 4) and top.dtype == torch.int32
    assert torch.ops.tdt_gb300.token_logprobs_backward(lp, ent, None, x, t, ent, stats, top).shape == x.shape
    with pytest.raises(NotImplementedError):  # CUDA kernels only: no silent CPU path
        autograd.token_logprobs(torch.zeros(6, 50), torch.zeros(6, dtype=torch.int64))
    for shape in ((3, 2), (6,), (2, 3, 1)):  # as many tokens, of other rows
        with pytest.raises(ValueError):
            autograd.token_logprobs(torch.zeros(2, 3, 50), torch.zeros(shape, dtype=torch.int64))
