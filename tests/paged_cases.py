"""Paged caches for the tests: pages in any order, entries and places past an utterance's end that may hold anything, and
the same rows as dense tensors in 64 bits."""
import math

import torch

E4M3 = torch.float8_e4m3fn
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.float16, torch.bfloat16]
NAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16", E4M3: "e4m3"}


def quantised(x):
    """Rows [..., D] as (values, bytes): the definition in 64 bits, on any device."""
    x = x.double()
    top = x.abs().amax(dim=-1)
    fine = x.isfinite().all(dim=-1)
    m, e = torch.frexp(torch.where(fine & (top > 0), top, 1.0))
    e = torch.where(m > 0.875, e - 8, e - 9)          # the least e with top <= 448 2^e = 0.875 2^(e + 9)
    e = torch.where(top > 0, e, -1000).clamp(-117, 120)
    y = torch.where(fine[..., None], x, 0.0) * torch.exp2(-e.double())[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    y = torch.round(y / step) * step                  # torch.round: ties to even
    value = torch.where(fine[..., None], y * torch.exp2(e.double())[..., None], math.nan)
    return value, torch.where(fine, e + 127, 255).to(torch.uint8)


def make(binding, lens, Hkv, D, page, dtype, seed=0, layout="plain", std=1.0, spread=0.0, room=0, poison=True):
    """(cache, page table, k, v): k, v in 64 bits [B, longest, Hkv, D], 0 past the utterances' ends.

    layout: "plain", "heads" (heads before places) or "fused" (k and v of a page side by side); spread: rows differ in size by up
    to 2^(+-spread); room: table columns more than needed."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, longest = len(lens), max(max(lens), 1)
    M = (longest + page - 1) // page + room
    need = [(n + page - 1) // page for n in lens]
    n_pages = sum(need) + 3
    shape = dict(plain=(n_pages, page, Hkv, D), heads=(n_pages, Hkv, page, D), fused=(n_pages, page, 2, Hkv, D))[layout]

    def tensors(shape, dt, value):
        if layout == "fused":
            base = torch.full(shape, value, device="cuda").to(dt)
            return base[:, :, 0], base[:, :, 1]
        two = [torch.full(shape, value, device="cuda").to(dt) for _ in range(2)]
        return [t.transpose(1, 2) for t in two] if layout == "heads" else two

    anything = math.nan if poison else 0.0
    pages = tensors(shape, dtype, anything)
    scales = [torch.full((n_pages, page, Hkv), 255 if poison else 127, dtype=torch.uint8, device="cuda") for _ in range(2)] \
        if dtype == E4M3 else [None, None]
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    junk = torch.tensor([-1, n_pages, -2 ** 31, 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda")
    table = junk[torch.randint(0, 5, (B, M), generator=g, device="cuda")]
    dense = [torch.zeros(B, longest, Hkv, D, dtype=torch.float64, device="cuda") for _ in range(2)]
    at = 0
    for b, n in enumerate(lens):
        mine = ids[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine
        if not n:
            continue
        pos = torch.arange(n, device="cuda")
        where = (mine.long()[pos // page], pos % page)
        for i in range(2):
            x = torch.randn(n, Hkv, D, generator=g, device="cuda") * std
            if spread:
                x *= torch.exp2((torch.rand(n, Hkv, 1, generator=g, device="cuda") * 2 - 1) * spread)
            if dtype == E4M3:
                x, byte = quantised(x)
                unit = torch.exp2(byte.double() - 127)[..., None]
                pages[i].view(torch.uint8)[where] = (x / unit).to(torch.float32).to(E4M3).view(torch.uint8)
                scales[i][where] = byte
            else:
                x = x.to(dtype)
                pages[i][where] = x
            dense[i][b, :n] = x.double()
    return (binding.PagedCache(*pages, *scales) if dtype == E4M3 else binding.PagedCache(*pages)), table, *dense


def i64(x):
    return torch.tensor(x, dtype=torch.int64, device="cuda")
