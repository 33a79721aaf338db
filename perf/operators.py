"""Cases of the attention and sampling operators: inputs, plain forms, exact values and the work that each case needs.

Cross attention of label states ``q`` [B, Lq, H, D] to encoder frames ``k``, ``v`` [B, Lk, Hkv, D] (``train``: forward and
backward; ``score``: forward only; ``step``: forward of a few rows, as in decoding), and ``sample``: drawing a token of each
row of logits from a given uniform number.  With ``own`` false ``run`` computes them with elementary torch operations in 32
bits, else with the package's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
ONE = 1 << 31  # the weight of a row's most probable token


def _attn(name, op, dtype, B, Lq, Lk, H, Hkv, D, ragged=False, window=0):
    return dict(name=name, op=op, dtype=dtype, B=B, Lq=Lq, Lk=Lk, H=H, Hkv=Hkv, D=D, ragged=ragged, window=window)


def _sample(name, dtype, N, V, width, per_row, temperature, top_k, top_p, min_p):
    return dict(name=name, op="sample", dtype=dtype, N=N, V=V, width=width, per_row=per_row, temperature=temperature,
                top_k=top_k, top_p=top_p, min_p=min_p)


def listed():
    return [
        # training an attention decoder over the encoder's frames, at the benchmark's batch of 4 x 200 frames x 40 labels
        _attn("train_4x41x200", "train", "bf16", 4, 41, 200, 8, 8, 64),
        # the large batch: 16 ragged utterances, 120 labels, 750 frames
        _attn("train_16x121x750_ragged", "train", "bf16", 16, 121, 750, 16, 16, 64, ragged=True),
        # the long utterance: 1,200 labels x 2,000 frames, in the 32 bits that its loss workload has
        _attn("train_1x1201x2000_f32", "train", "f32", 1, 1201, 2000, 8, 8, 64),
        # long labels whose queries see only frames near their transducer alignment; heads share keys; an odd head width
        _attn("train_8x1201x2000_window", "train", "f16", 8, 1201, 2000, 8, 2, 96, ragged=True, window=300),
        # the largest training call: packed long-form batches, four query heads to a key head
        _attn("train_16x1024x4096_gqa", "train", "bf16", 16, 1024, 4096, 16, 4, 128),
        # rescoring hypotheses over long recordings: forward only
        _attn("score_8x121x7501", "score", "bf16", 8, 121, 7501, 16, 4, 128, ragged=True),
        # one decoding step of one utterance: the smallest call
        _attn("step_1x1x200", "step", "bf16", 1, 1, 200, 8, 8, 64),
        # one decoding step of a ragged batch
        _attn("step_64x1x750_ragged", "step", "f16", 64, 1, 750, 16, 16, 64, ragged=True),
        # one decoding step of a server's batch over long recordings
        _attn("step_128x1x6000_gqa", "step", "bf16", 128, 1, 6000, 32, 8, 128),
        # drawing one token of the benchmark's vocabulary
        _sample("sample_1x8193", "f32", 1, 8193, 8193, False, 0.8, 50, 0.95, 0.0),
        # the token logits of joint outputs [..., :8193] in place, each row with its request's own settings
        _sample("sample_656x8193_rows", "f32", 656, 8193, 8198, True, 0.9, 100, 0.9, 0.02),
        # a server's batch over a wide vocabulary, nucleus sampling
        _sample("sample_2048x131072", "bf16", 2048, 131072, 131072, False, 0.7, 0, 0.9, 0.0),
    ]


MOST_PAIRS = {"train": 16 * 1024 * 4096 * 16 * 128, "score": 8 * 121 * 7501 * 16 * 128, "step": 128 * 6000 * 32 * 128}


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["train", "train", "score", "step", "step", "sample", "sample"])
    if op == "sample":
        V = _spread(rng, 40, 131072)
        N = max(1, min(_spread(rng, 1, 4096), 2048 * 131072 // V // 2))
        return dict(op=op, dtype=rng.choice(["f32", "f16", "bf16"]), N=N, V=V, width=V + rng.choice([0, 0, 3, 5, 8]),
                    per_row=rng.random() < 0.4, temperature=round(rng.uniform(0.3, 1.3), 2),
                    top_k=rng.choice([0, 0, 1, 5, 40, 50, 200, 1000]), top_p=rng.choice([1.0, 1.0, 0.95, 0.9, 0.5]),
                    min_p=rng.choice([0.0, 0.0, 0.05, 0.1]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    D = rng.choice([64, 64, 128, 128, 80, 96, 40])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4])
    Lq = _spread(rng, 1, 8) if op == "step" else _spread(rng, 9, 1500)
    Lk = _spread(rng, 20, 8000)
    B = _spread(rng, 1, 128 if op == "step" else 32)
    most = MOST_PAIRS[op] // (8 if dtype == "f32" else 1)
    B = max(1, min(B, most // (Lq * Lk * H * D)))
    return dict(op=op, dtype=dtype, B=B, Lq=Lq, Lk=Lk, H=H, Hkv=Hkv, D=D, ragged=rng.random() < 0.5,
                window=rng.choice([0, 0, 0, _spread(rng, 10, 1000)]) if op == "train" else 0)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dt)

    if case["op"] == "sample":
        N, V = case["N"], case["V"]
        s = dict(case=case, logits=randn(N, case["width"], std=3.0)[:, :V],
                 u=torch.rand(N, generator=g, device=dev))
        for key in ("temperature", "top_k", "top_p", "min_p"):
            s[key] = case[key]
        if case["per_row"]:
            f = torch.rand(4, N, generator=g, device=dev)
            s["temperature"] = case["temperature"] * (0.5 + f[0])
            s["top_k"] = (case["top_k"] * 2 * f[1]).to(torch.int32)
            s["top_p"] = 1.0 - (1.0 - case["top_p"]) * f[2]
            s["min_p"] = case["min_p"] * 2 * f[3]
        return s
    B, Lq, Lk, H, Hkv, D = (case[x] for x in ("B", "Lq", "Lk", "H", "Hkv", "D"))
    q = randn(B, Lq, H, D, std=1.5)
    kv = randn(B, Lk, 2, Hkv, D)  # one projection of the frames gives both
    s = dict(case=case, q=q, k=kv[:, :, 0], v=kv[:, :, 1], k_lens=None, q_lens=None, windows=None)
    if case["ragged"]:
        s["k_lens"] = torch.randint((Lk + 1) // 2, Lk + 1, (B,), generator=g, device=dev)
        if case["op"] != "step":
            s["q_lens"] = torch.randint((Lq + 1) // 2, Lq + 1, (B,), generator=g, device=dev)
    if case["window"]:
        w = case["window"]
        at = (torch.rand(B, Lq, generator=g, device=dev).sort(dim=1).values * Lk).to(torch.int32)
        s["windows"] = torch.stack([at - w // 2, at + w - w // 2], dim=-1)
    if case["op"] == "train":
        s["grad_out"] = randn(B, Lq, H, D)
    return s


# ---------------------------------------------------------------- plain forms


def _seen(s, dev):
    """[B, Lq, Lk] truth values: the frames that each query sees."""
    c = s["case"]
    B, Lq, Lk = c["B"], c["Lq"], c["Lk"]
    j = torch.arange(Lk, device=dev)
    m = torch.ones(B, Lq, Lk, dtype=torch.bool, device=dev)
    if s["k_lens"] is not None:
        m &= (j < s["k_lens"][:, None])[:, None]
    if s["q_lens"] is not None:
        m &= (torch.arange(Lq, device=dev) < s["q_lens"][:, None])[..., None]
    if s["windows"] is not None:
        w = s["windows"].to(torch.int64)
        m &= (j >= w[..., :1]) & (j < w[..., 1:])
    return m


def _heads(x, Hkv):
    """[B, L, H, D] as [B, Hkv, H / Hkv * L, D], in 32 bits."""
    B, L, H, D = x.shape
    return x.float().reshape(B, L, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)


def _back(x, L, dtype):
    B, Hkv, R, D = x.shape
    return x.reshape(B, Hkv, R // L, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, Hkv * (R // L), D).to(dtype)


def _plain_attn(s):
    c = s["case"]
    Hkv, Lq, Lk, D = c["Hkv"], c["Lq"], c["Lk"], c["D"]
    G, dt, scale = c["H"] // Hkv, s["q"].dtype, 1.0 / math.sqrt(D)
    q, k, v = _heads(s["q"], Hkv), _heads(s["k"], Hkv), _heads(s["v"], Hkv)
    seen = _seen(s, q.device)[:, None, None].expand(-1, 1, G, -1, -1).reshape(c["B"], 1, G * Lq, Lk)
    x = torch.where(seen, torch.matmul(q, k.transpose(2, 3)) * scale, -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    del x
    total = p.sum(dim=-1, keepdim=True)
    p /= torch.where(total > 0, total, 1.0)
    o = torch.matmul(p, v)
    if c["op"] != "train":
        return _back(o, Lq, dt)
    do = _heads(s["grad_out"], Hkv)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds -= (do * o).sum(dim=-1, keepdim=True)
    ds *= p
    ds *= scale
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    return dict(out=_back(o, Lq, dt), dq=_back(dq, Lq, dt), dk=_back(dk, Lk, dt), dv=_back(dv, Lk, dt))


def _column(x, like, dtype):
    """A setting of all rows, or of each, as a column."""
    if isinstance(x, torch.Tensor):
        return x.to(dtype)[:, None]
    return torch.full((like.shape[0], 1), x, dtype=dtype, device=like.device)


def _share(total, part24):
    """floor(total * part24 / 2^24) of whole numbers, exactly."""
    return (total >> 24) * part24 + (((total & 0xFFFFFF) * part24) >> 24)


def _plain_sample(s):
    x = s["logits"].float()
    N, V = x.shape
    T = _column(s["temperature"], x, torch.float32)
    k = _column(s["top_k"], x, torch.int64)
    p24 = torch.round(_column(s["top_p"], x, torch.float32) * 2.0**24).to(torch.int64)
    m = torch.ceil(_column(s["min_p"], x, torch.float32) * 2.0**31).to(torch.int64)
    u24 = (s["u"] * 2.0**24).to(torch.int64)[:, None].clamp(0, (1 << 24) - 1)
    xs, at = torch.sort(x, dim=-1, descending=True, stable=True)
    top = xs[:, :1]
    per = torch.full_like(T, math.log2(math.e)) / T
    w = torch.round(torch.exp2((xs - top) * per) * 2.0**31).to(torch.int64)  # of the sorted row; whole numbers: sums are exact
    rank = torch.arange(V, device=x.device)
    w = torch.where((rank < k) | (k <= 0), w, 0)
    run = torch.cumsum(w, dim=-1)
    stays = (run - w < _share(run[:, -1:], p24)) | (p24 >= 1 << 24)
    w = torch.where((stays & (w >= m)) | (rank == 0), w, 0)
    w = torch.zeros_like(w).scatter_(1, at, w)  # back in the vocabulary's order
    run = torch.cumsum(w, dim=-1)
    total = run[:, -1:]
    token = (run > _share(total, u24)).to(torch.int8).argmax(dim=-1, keepdim=True)
    logp = (x.gather(1, token) - top) / T - torch.log(total.float() / 2.0**31)
    return dict(tokens=token[:, 0].to(torch.int32), logprobs=logp[:, 0])


def run(s):
    if not own:
        return _plain_sample(s) if s["case"]["op"] == "sample" else _plain_attn(s)
    from transducer_loss_asr_gb300 import binding

    if s["case"]["op"] == "sample":
        tokens, logprobs = binding.tdt_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
        return dict(tokens=tokens, logprobs=logprobs)
    sees = dict(k_lens=s["k_lens"], q_lens=s["q_lens"], windows=s["windows"])
    if s["case"]["op"] != "train":
        return binding.tdt_cross_attn_fwd(s["q"], s["k"], s["v"], need_lse=False, **sees)[0]
    out, lse = binding.tdt_cross_attn_fwd(s["q"], s["k"], s["v"], **sees)
    dq, dk, dv = binding.tdt_cross_attn_bwd(s["grad_out"], s["q"], s["k"], s["v"], out, lse, **sees)
    return dict(out=out, dq=dq, dk=dk, dv=dv)


# ---------------------------------------------------------------- the work and the values


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "sample":
        n = case["N"] * case["V"]
        return {"bytes": n * e + case["N"] * (4 + 8 + (16 if case["per_row"] else 0)), "flops": 4 * n}
    B, Lq, Lk, H, Hkv, D = (case[x] for x in ("B", "Lq", "Lk", "H", "Hkv", "D"))
    # lengths are uniform in [L / 2, L]; what no query sees is not read, and gradients are written whole
    fk = 0.75 if case["ragged"] else 1.0
    fq = 0.75 if case["ragged"] and case["op"] != "step" else 1.0
    keys = fk * Lk if not case["window"] else min(fk * Lk, case["window"])
    pairs = B * H * fq * Lq * keys
    qs, ks = B * Lq * H * D * e, B * Lk * Hkv * D * e
    if case["op"] == "train":
        return {"bytes": fq * 2 * qs + 2 * qs + fk * 2 * ks + 2 * ks, "flops": 14 * D * pairs}
    return {"bytes": fq * qs + qs + fk * 2 * ks, "flops": 4 * D * pairs}


def _exact_attn(case, s):
    B, Lq, Lk, H, Hkv, D = (case[x] for x in ("B", "Lq", "Lk", "H", "Hkv", "D"))
    train = case["op"] == "train"
    out = {n: torch.zeros(B, Lk if n in ("dk", "dv") else Lq, Hkv if n in ("dk", "dv") else H, D, dtype=torch.float64,
                          device=s["q"].device) for n in (("out", "dq", "dk", "dv") if train else ("out",))}
    for b in range(B):
        nk = Lk if s["k_lens"] is None else int(s["k_lens"][b])
        nq = Lq if s["q_lens"] is None else int(s["q_lens"][b])
        for h in range(H):
            c = h // (H // Hkv)
            q, k, v = s["q"][b, :nq, h].double(), s["k"][b, :nk, c].double(), s["v"][b, :nk, c].double()
            x = torch.einsum("id,jd->ij", q, k) / D**0.5
            if s["windows"] is not None:
                w, j = s["windows"][b, :nq], torch.arange(nk, device=q.device)[None]
                x = x.masked_fill((j < w[:, :1]) | (j >= w[:, 1:]), -1e300)
                some = ((w[:, 1].clamp(max=nk) - w[:, 0].clamp(min=0)) > 0)[:, None]
            p = torch.softmax(x, dim=1)
            if s["windows"] is not None:
                p = p * some
            o = torch.einsum("ij,jd->id", p, v)
            out["out"][b, :nq, h] = o
            if train:
                g = s["grad_out"][b, :nq, h].double()
                d = p * (torch.einsum("id,jd->ij", g, v) - torch.einsum("id,id->i", g, o)[:, None]) / D**0.5
                out["dq"][b, :nq, h] = torch.einsum("ij,jd->id", d, k)
                out["dk"][b, :nk, c] += torch.einsum("ij,id->jd", d, q)
                out["dv"][b, :nk, c] += torch.einsum("ij,id->jd", p, g)
    return out if train else out["out"]


def _exact_sample(case, s):
    """log-probability of the drawn token; the draw itself is a whole number."""
    N, V = case["N"], case["V"]
    logp = torch.empty(N, dtype=torch.float64, device=s["u"].device)

    def of(key, i):
        return s[key][i].item() if isinstance(s[key], torch.Tensor) else s[key]

    for i in range(N):
        x = s["logits"][i].double()
        z = (x - x.max()) / of("temperature", i)
        w = (z.exp() * ONE).round().long()
        order = torch.argsort(x, descending=True, stable=True)
        if of("top_k", i) > 0:
            order = order[: of("top_k", i)]
        ws = w[order]
        p = of("top_p", i)
        if p < 1:
            before = ws.cumsum(0) - ws
            ws, order = (t[(before < int(int(ws.sum()) * round(p * 2**24)) >> 24) | (before == 0)] for t in (ws, order))
        stay = ws >= math.ceil(of("min_p", i) * ONE)
        stay[0] = True
        order = order[stay].sort().values
        run = w[order].cumsum(0)
        at = int((run > (int(run[-1]) * int(float(s["u"][i]) * 2**24)) >> 24).to(torch.int8).argmax())
        logp[i] = z[order[at]] - torch.log(torch.exp(z[order]).sum())
    return dict(tokens=None, logprobs=logp)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    return _exact_attn(case, s)
