"""Cases of the label-cache and scoring operators: inputs, plain forms, exact values and the work that each case needs.

An attention decoder keeps the keys and values of its label states in pages, ``write``: new rows go into pages of their own type,
``store``: new rows are quantised as they are written (e4m3 and a power of two a row) and read back; ``step`` and ``chunk``: one or
many new label states of each hypothesis read its pages, causally.  Its logits are turned into log-probabilities of given tokens,
with the entropy of each row: ``score`` (forward, with the most probable alternatives), ``grad`` (forward, then backward) and
``train`` (both in one call).  With ``own`` false ``run`` computes them with elementary torch operations in 32 bits, else with the
package's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


def _cache(name, op, dtype, cache, B, Lq, past, H, Hkv, D, page, ragged=False):
    return dict(name=name, op=op, dtype=dtype, cache=cache, B=B, Lq=Lq, past=past, H=H, Hkv=Hkv, D=D, page=page, ragged=ragged)


def _rows(name, op, dtype, N, V, width, n_top=0, padded=False, banned=False):
    return dict(name=name, op=op, dtype=dtype, N=N, V=V, width=width, n_top=n_top, padded=padded, banned=banned)


def listed():
    return [
        # a decoding step's keys and values of a ragged batch of 64 hypotheses go into their pages as they are
        _cache("write_64x1x750", "write", "f16", "f16", 64, 1, 750, 16, 16, 64, 32, ragged=True),
        # the benchmark's 4 utterances of 40 labels, quantised: what a beam of hypotheses starts from
        _cache("store_4x41_e4m3", "store", "bf16", "e4m3", 4, 41, 0, 8, 8, 64, 16),
        # packed long-form label sequences, quantised and read back
        _cache("store_16x1024_e4m3", "store", "bf16", "e4m3", 16, 1024, 1024, 16, 4, 128, 64, ragged=True),
        # one decoding step of one hypothesis of 41 labels: the smallest call
        _cache("step_1x1x40", "step", "bf16", "bf16", 1, 1, 40, 8, 8, 64, 16),
        # one decoding step of a ragged batch
        _cache("step_64x1x750_ragged", "step", "f16", "f16", 64, 1, 750, 16, 16, 64, 32, ragged=True),
        # one decoding step of a server's batch over long quantised caches, four query heads to a key head
        _cache("step_128x1x6000_e4m3", "step", "bf16", "e4m3", 128, 1, 6000, 32, 8, 128, 64),
        # rescoring: 120 labels more of 16 ragged hypotheses
        _cache("chunk_16x121x750_ragged", "chunk", "bf16", "bf16", 16, 121, 750, 16, 16, 64, 16, ragged=True),
        # a long prompt behind long quantised caches: the largest call
        _cache("chunk_8x1024x7168_e4m3", "chunk", "bf16", "e4m3", 8, 1024, 7168, 16, 4, 128, 64),
        # the score of one drawn token of the benchmark's vocabulary, with ten alternatives
        _rows("score_1x8193", "score", "f32", 1, 8193, 8193, n_top=10),
        # confidences of a server's batch over a wide vocabulary in which some tokens are not allowed
        _rows("score_2048x131072", "score", "bf16", 2048, 131072, 131072, n_top=20, banned=True),
        # training on the token logits of joint outputs [..., :8193] in place; padded label rows
        _rows("grad_656x8193", "grad", "f32", 656, 8193, 8198, padded=True),
        # training a decoder of a wide vocabulary: log-probabilities and gradient in one call
        _rows("train_4096x50257", "train", "bf16", 4096, 50257, 50257, padded=True),
    ]


MOST_PAIRS = {"chunk": 8 * 1024 * 7168 * 16 * 128, "step": 128 * 6000 * 32 * 128, "store": 16 * 1024 * 16 * 128, "write": 64 * 750 * 16 * 64}


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "store", "store", "step", "step", "step", "chunk", "chunk", "chunk", "score", "score", "grad", "train"])
    if op in ("score", "grad", "train"):
        V = _spread(rng, 40, 131072)
        N = max(1, min(_spread(rng, 1, 4096), 2048 * 131072 // V // (2 if op == "score" else 4)))
        return dict(op=op, dtype=rng.choice(["f32", "f16", "bf16"]), N=N, V=V, width=V + rng.choice([0, 0, 3, 5, 8]),
                    n_top=rng.choice([0, 1, 5, 10, 32]) if op == "score" else 0, padded=rng.random() < 0.5, banned=rng.random() < 0.3)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    D = rng.choice([64, 64, 128, 128, 80, 96, 40])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4])
    Lq = _spread(rng, 1, 8) if op in ("step", "write") else _spread(rng, 9, 1500)
    past = _spread(rng, 1, 8000)
    B = _spread(rng, 1, 128 if op in ("step", "write") else 32)
    most = MOST_PAIRS[op] // (8 if dtype == "f32" and op == "chunk" else 1)
    each = {"write": (Lq + past) * Hkv * D, "store": Lq * H * D}.get(op, Lq * past * H * D)
    return dict(op=op, dtype=dtype, cache=dtype if op == "write" else "e4m3" if op == "store" else rng.choice([dtype, "e4m3"]),
                B=max(1, min(B, most // each)), Lq=Lq, past=past, H=H, Hkv=Hkv, D=D, page=rng.choice([8, 16, 16, 32, 64, 128, 256]),
                ragged=rng.random() < 0.5)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dt)

    if case["op"] in ("score", "grad", "train"):
        N, V = case["N"], case["V"]
        x = randn(N, case["width"], std=3.0)
        tokens = torch.randint(0, V, (N,), generator=g, device=dev)
        if case["banned"]:  # tokens that may not follow: about one in 16
            x.masked_fill_(torch.randint(0, 16, x.shape, generator=g, device=dev, dtype=torch.uint8) == 0, -math.inf)
            x[torch.arange(N, device=dev), tokens] = 1.0
        if case["padded"]:
            tokens.masked_fill_(torch.rand(N, generator=g, device=dev) < 0.25, -100)
        s = dict(case=case, logits=x[:, :V], tokens=tokens)
        if case["op"] != "score":  # a mean over the labels, with a little weight on the entropy
            s["grad_logprobs"] = -(0.5 + torch.rand(N, generator=g, device=dev)) / N
            s["grad_entropy"] = -0.1 * torch.rand(N, generator=g, device=dev) / N
        return s
    B, Lq, past, H, Hkv, D, P = (case[x] for x in ("B", "Lq", "past", "H", "Hkv", "D", "page"))
    qkv = randn(B, Lq, H + 2 * Hkv, D, std=1.5)  # one projection of the label states gives all three
    s = dict(case=case, q=qkv[:, :, :H], k=qkv[:, :, H:H + Hkv], v=qkv[:, :, H + Hkv:], q_lens=None)
    s["kv_lens"] = torch.full((B,), past + Lq, dtype=torch.int64, device=dev)
    if case["ragged"]:
        s["kv_lens"] = torch.randint((past + 1) // 2, past + 1, (B,), generator=g, device=dev) + Lq
        if Lq > 8:
            s["q_lens"] = torch.randint((Lq + 1) // 2, Lq + 1, (B,), generator=g, device=dev)
            s["kv_lens"] += s["q_lens"] - Lq
    M = (past + Lq + P - 1) // P  # pages of an utterance, in any order; entries past its end name none
    table = torch.randperm(B * M, generator=g, device=dev).view(B, M).to(torch.int32)
    s["page_table"] = table.masked_fill_(torch.arange(M, device=dev) * P >= s["kv_lens"][:, None], -1)
    for n in "kv":
        x = randn(B * M, P, Hkv, D)
        s[n + "_scales"] = None
        if case["cache"] == "e4m3":
            x, s[n + "_scales"] = _quantised(x.float())
        s[n + "_pages"] = x
    return s


# ---------------------------------------------------------------- plain forms


def _quantised(x):
    """Rows [..., D] in 32 bits as e4m3 and one byte each: x = e4m3 2^(byte - 127), the power of two the least that keeps the
    row's largest element within 448."""
    m, e = torch.frexp(x.abs().amax(dim=-1))
    byte = (torch.where(m > 0.875, e - 8, e - 9).clamp(-117, 120) + 127).to(torch.int32)
    down = ((254 - byte) << 23).view(torch.float32)
    return (x * down[..., None]).to(torch.float8_e4m3fn), byte.to(torch.uint8)


def _values(pages, scales):
    if scales is None:
        return pages.float()
    return pages.float() * (scales.to(torch.int32) << 23).view(torch.float32)[..., None]


def _places(s):
    """Where the new rows go, [B, Lq]: their positions, which of them take part, pages and places in these."""
    c = s["case"]
    at = torch.arange(c["Lq"], device=s["q"].device)
    n = torch.full_like(s["kv_lens"], c["Lq"]) if s["q_lens"] is None else s["q_lens"]
    pos = (s["kv_lens"] - n)[:, None] + at
    real = at < n[:, None]
    page = s["page_table"].gather(1, torch.where(real, pos, 0) // c["page"]).long()
    return pos, real, page, pos % c["page"]


def _plain_write(s):
    _, real, page, slot = _places(s)
    page, slot = page[real], slot[real]
    for n in "kv":
        x = s[n][real]
        if s[n + "_scales"] is not None:
            x, s[n + "_scales"][page, slot] = _quantised(x.float())
        s[n + "_pages"][page, slot] = x


def _plain_read(s):
    _, real, page, slot = _places(s)
    page = page.clamp_min(0)
    out = {}
    for n in "kv":
        scales = s[n + "_scales"]
        x = _values(s[n + "_pages"][page, slot], None if scales is None else scales[page, slot])
        out[n] = torch.where(real[..., None, None], x, 0.0).to(s[n].dtype)
    return out


def _plain_attn(s):
    c = s["case"]
    B, Lq, H, Hkv, D = (c[x] for x in ("B", "Lq", "H", "Hkv", "D"))
    G, Lk = H // Hkv, c["past"] + Lq
    table = s["page_table"].clamp_min(0).long()

    def whole(n):  # [B, Hkv, Lk, D]
        scales = s[n + "_scales"]
        x = _values(s[n + "_pages"][table], None if scales is None else scales[table])
        return x.flatten(1, 2)[:, :Lk].transpose(1, 2)

    k, v = whole("k"), whole("v")
    q = s["q"].float().reshape(B, Lq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Lq, D)
    pos, real, _, _ = _places(s)
    seen = (torch.arange(Lk, device=q.device) <= pos[..., None]) & real[..., None]
    seen = seen[:, None, None].expand(-1, 1, G, -1, -1).reshape(B, 1, G * Lq, Lk)
    x = torch.where(seen, torch.matmul(q, k.transpose(2, 3)) / math.sqrt(D), -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o.reshape(B, Hkv, G, Lq, D).permute(0, 3, 1, 2, 4).reshape(B, Lq, H, D).to(s["q"].dtype)


def _plain_rows(s):
    c = s["case"]
    x, tokens = s["logits"].float(), s["tokens"]
    real = tokens >= 0  # labels of -100 are padding: their rows take no part
    x = x - x.amax(dim=-1, keepdim=True)
    lp = x - torch.log(torch.exp(x).sum(dim=-1, keepdim=True))
    p = torch.exp(lp)
    ent = torch.where(real, -(p * torch.where(p > 0, lp, 0.0)).sum(dim=-1), 0.0)
    given = tokens.clamp_min(0)[:, None]
    out = dict(logprobs=torch.where(real, lp.gather(1, given)[:, 0], 0.0), entropy=ent)
    if c["n_top"]:
        top, at = torch.sort(s["logits"], dim=-1, descending=True, stable=True)  # ties: the lowest token first
        at = at[:, :c["n_top"]]
        out["top_tokens"] = torch.where(real[:, None], at, -1).to(torch.int32)
        out["top_logprobs"] = torch.where(real[:, None], lp.gather(1, at), -math.inf)
    if c["op"] != "score":
        a, b = s["grad_logprobs"][:, None], s["grad_entropy"][:, None]
        grad = -p * (a + b * (torch.where(p > 0, lp, 0.0) + ent[:, None]))
        grad.scatter_add_(1, given, a)
        out["grad"] = torch.where(real[:, None], grad, 0.0).to(s["logits"].dtype)
    return out


def run(s):
    op = s["case"]["op"]
    if own:
        from transducer_loss_asr_gb300 import binding

        if op == "score":
            r = binding.tdt_token_logprobs_fwd(s["logits"], s["tokens"], n_top=s["case"]["n_top"])
            out = dict(logprobs=r.logprobs, entropy=r.entropy)
            return dict(out, top_tokens=r.top_tokens, top_logprobs=r.top_logprobs) if s["case"]["n_top"] else out
        if op == "grad":
            r = binding.tdt_token_logprobs_fwd(s["logits"], s["tokens"])
            grad = binding.tdt_token_logprobs_bwd(s["logits"], s["tokens"], r, s["grad_logprobs"], s["grad_entropy"])
            return dict(logprobs=r.logprobs, entropy=r.entropy, grad=grad)
        if op == "train":
            r, grad = binding.tdt_token_logprobs_fwd_bwd(s["logits"], s["tokens"], s["grad_logprobs"], s["grad_entropy"])
            return dict(logprobs=r.logprobs, entropy=r.entropy, grad=grad)
        cache = binding.PagedCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        if op in ("write", "store"):
            binding.tdt_cache_write(s["k"], s["v"], cache, s["page_table"], s["kv_lens"], s["q_lens"])
            if op == "write":
                return dict(k=s["k_pages"], v=s["v_pages"])
            k, v = binding.tdt_cache_read(cache, s["page_table"], s["kv_lens"], s["q_lens"], s["case"]["Lq"], s["k"].dtype)
            return dict(k=k, v=v)
        return binding.tdt_paged_attn(s["q"], cache, s["page_table"], s["kv_lens"], s["q_lens"])[0]
    if op in ("score", "grad", "train"):
        return _plain_rows(s)
    if op in ("write", "store"):
        _plain_write(s)
        return dict(k=s["k_pages"], v=s["v_pages"]) if op == "write" else _plain_read(s)
    return _plain_attn(s)


# ---------------------------------------------------------------- the work and the values


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("score", "grad", "train"):
        N, n = case["N"], case["N"] * case["V"]
        part = 0.75 if case["padded"] else 1.0  # rows that take part; gradients are written whole
        if case["op"] == "score":
            return {"bytes": part * n * e + N * (8 + 8 + 8 * case["n_top"]), "flops": part * 6 * n}
        return {"bytes": part * n * e + n * e + N * (8 + 8 + 8), "flops": part * 10 * n}
    B, Lq, past, H, Hkv, D = (case[x] for x in ("B", "Lq", "past", "H", "Hkv", "D"))
    # lengths are uniform in [L / 2, L]
    fp = 0.75 if case["ragged"] else 1.0
    fq = 0.75 if case["ragged"] and Lq > 8 else 1.0
    rows = B * Lq * Hkv * 2  # of k and v
    row = D * BYTES[case["cache"]] + (1 if case["cache"] == "e4m3" else 0)
    if case["op"] == "write":
        return {"bytes": fq * rows * (D * e + row), "flops": 0}
    if case["op"] == "store":  # written from D e bytes a row, and read back to as many
        return {"bytes": fq * rows * (D * e + row) + fq * rows * row + rows * D * e, "flops": fq * rows * 4 * D}
    pairs = B * H * (fq * Lq * fp * past + (fq * Lq) ** 2 / 2 + fq * Lq / 2)
    return {"bytes": (fq + 1) * B * Lq * H * D * e + B * 2 * Hkv * (fp * past + fq * Lq) * row, "flops": 4 * D * pairs}


def _grid(x):
    """e4m3's rounding in 64 bits of rows within 448: steps of 2^-3 of the power of two below, 2^-9 at the least; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_rows(case, s):
    N, V = case["N"], case["V"]
    dev = s["logits"].device
    out = dict(logprobs=torch.zeros(N, dtype=torch.float64, device=dev), entropy=torch.zeros(N, dtype=torch.float64, device=dev))
    if case["n_top"]:
        out |= dict(top_tokens=None, top_logprobs=torch.full((N, case["n_top"]), -math.inf, dtype=torch.float64, device=dev))
    if case["op"] != "score":
        out["grad"] = torch.zeros(N, V, dtype=torch.float64, device=dev)
    for i in range(0, N, 256):
        x, t = s["logits"][i:i + 256].double(), s["tokens"][i:i + 256]
        rows = torch.nonzero(t >= 0)[:, 0]
        x, t = x[rows], t[rows]
        lp = x - torch.logsumexp(x, dim=1, keepdim=True)
        p = torch.softmax(x, dim=1)
        h = -torch.special.xlogy(p, p).sum(dim=1)
        at = torch.arange(len(rows), device=dev)
        out["logprobs"][i + rows], out["entropy"][i + rows] = lp[at, t], h
        if case["n_top"]:
            out["top_logprobs"][i + rows] = lp.topk(case["n_top"], dim=1).values
        if case["op"] != "score":
            a, b = s["grad_logprobs"][i + rows].double(), s["grad_entropy"][i + rows].double()
            d = -p * a[:, None] - b[:, None] * (torch.special.xlogy(p, p) + p * h[:, None])
            d[at, t] += a
            out["grad"][i + rows] = d
    return out


def _utterance(s, b, n):
    """(first new position, one past the last, rows [Hkv, positions, D] of the cache) of utterance b, in 64 bits."""
    c = s["case"]
    end = int(s["kv_lens"][b])
    new = c["Lq"] if s["q_lens"] is None else int(s["q_lens"][b])
    pages = s["page_table"][b, :(end + c["page"] - 1) // c["page"]].long()
    x = s[n + "_pages"][pages].double()
    if s[n + "_scales"] is not None:
        x = x * torch.exp2(s[n + "_scales"][pages].double() - 127)[..., None]
    return end - new, end, x.flatten(0, 1)[:end].transpose(0, 1)


def _exact_cache(case, s):
    B, Lq, P = case["B"], case["Lq"], case["page"]
    out = {n: (s[n + "_pages"] if case["op"] == "write" else torch.zeros_like(s[n])).double() for n in "kv"}
    for n in "kv":
        for b in range(B):
            first, end, _ = _utterance(s, b, n)
            x = s[n][b, :end - first].double()
            if case["op"] == "write":
                pos = torch.arange(first, end, device=x.device)
                out[n][s["page_table"][b, pos // P].long(), pos % P] = x
            else:
                top = x.abs().amax(dim=-1, keepdim=True)
                unit = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-117, 120))
                out[n][b, :end - first] = _grid(x / unit) * unit
    return out


def _exact_attn(case, s):
    B, H, G = case["B"], case["H"], case["H"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        first, end, k = _utterance(s, b, "k")
        v = _utterance(s, b, "v")[2]
        later = torch.arange(end, device=k.device) > torch.arange(first, end, device=k.device)[:, None]
        for h in range(H):
            x = s["q"][b, :end - first, h].double() @ k[h // G].T / case["D"] ** 0.5
            out[b, :end - first, h] = torch.softmax(x.masked_fill_(later, -1e300), dim=1) @ v[h // G]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("score", "grad", "train"):
        return _exact_rows(case, s)
    return _exact_cache(case, s) if case["op"] in ("write", "store") else _exact_attn(case, s)
