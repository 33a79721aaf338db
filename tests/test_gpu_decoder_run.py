"""The label cache, its attention, sampling and scoring together, as a decoding loop uses them, against plain arithmetic in 64 bits."""
import pytest
import torch

from paged_cases import E4M3, i64, quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transducer_loss_asr_gb300 import binding as b

    return b


N, STEPS, H, K, D, PAGE, VOCAB = 6, 37, 4, 2, 64, 8, 500


def _projections(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    embed = torch.randn(VOCAB, (H + 2 * K) * D, generator=g, device="cuda").to(torch.bfloat16)
    vocab = (torch.randn(H * D, VOCAB, generator=g, device="cuda") / 4).to(torch.bfloat16)
    uniforms = torch.rand(STEPS, N, generator=g, device="cuda")
    return embed, vocab, uniforms


def _heads(embed, tokens):
    x = embed[tokens].view(*tokens.shape, H + 2 * K, D)
    return x[:, :, :H], x[:, :, H:H + K], x[:, :, H + K:]


def _loop(binding, embed, vocab, uniforms, cache, table, lens, graph):
    """The decoding loop: tokens [N, STEPS + 1], attention outputs, log-probabilities, entropies; captured or not."""
    tokens = torch.arange(N, device="cuda").view(N, 1)
    state = dict(tokens=tokens.clone(), u=torch.empty(N, device="cuda"))

    def step():
        lens.add_(1)
        q, k, v = _heads(embed, state["tokens"])
        binding.tdt_cache_write(k, v, cache, table, lens)
        out, _ = binding.tdt_paged_attn(q, cache, table, lens)
        logits = out.flatten(1) @ vocab
        drawn, _ = binding.tdt_sample(logits, state["u"], temperature=0.9, top_k=40)
        r = binding.tdt_token_logprobs_fwd(logits, drawn.long(), n_top=3)
        state["tokens"].copy_(drawn.view(N, 1))
        return out, logits, r

    results, history = [], [tokens]
    captured = None
    if graph:
        lens.zero_()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            state["u"].copy_(uniforms[0])
            step()
        torch.cuda.current_stream().wait_stream(s)
        lens.zero_()
        state["tokens"].copy_(tokens)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            kept = step()
    for i in range(STEPS):
        state["u"].copy_(uniforms[i])
        if graph:
            captured.replay()
            got = kept
        else:
            got = step()
        results.append((got[0].clone(), got[1].clone(), tuple(t.clone() for t in got[2])))
        history.append(state["tokens"].clone())
    return torch.cat(history, 1), results


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_decoding_loop_and_rescoring(binding, cache_dtype):
    embed, vocab, uniforms = _projections(3)
    pages = (STEPS + PAGE - 1) // PAGE
    cache = binding.PagedCache.empty(N * pages, PAGE, K, D, cache_dtype)
    table = torch.randperm(N * pages, device="cuda").view(N, pages).to(torch.int32)
    lens = i64([0] * N)
    tokens, results = _loop(binding, embed, vocab, uniforms, cache, table, lens, False)
    again, captured = _loop(binding, embed, vocab, uniforms, cache, table, i64([0] * N), True)
    assert torch.equal(tokens, again)
    for a, b in zip(results, captured):
        assert torch.equal(a[0], b[0]) and all(torch.equal(x, y) for x, y in zip(a[2], b[2]))
    # in 64 bits, from the tokens that were drawn
    q, k, v = _heads(embed, tokens[:, :-1])
    k, v = (quantised(t)[0] if cache_dtype == E4M3 else t.double() for t in (k, v))
    read = binding.tdt_cache_read(cache, table, lens, lens, STEPS, torch.float32)
    assert torch.equal(read[0].double(), k) and torch.equal(read[1].double(), v)
    k, v = (t.repeat_interleave(H // K, 2).transpose(1, 2) for t in (k, v))
    s = q.double().transpose(1, 2) @ k.transpose(2, 3) * D ** -0.5
    s = s.masked_fill(torch.ones(STEPS, STEPS, dtype=torch.bool, device="cuda").triu(1), -1e300)
    p = torch.softmax(s, 3)
    out = (p @ v).transpose(1, 2)
    # weights and results are rounded to bfloat16 (half a step: 2^-9 of a value in [1, 2), 2^-8 relative at most); float32's part is
    # far below
    bound = (2.0 ** -8 * (p @ v.abs())).transpose(1, 2) + 2.0 ** -8 * out.abs() + 1e-4
    for i, (got, logits, r) in enumerate(results):
        assert bool(((got[:, 0].double() - out[:, i]).abs() <= bound[:, i]).all())
        lp = torch.log_softmax(logits.double(), 1)
        drawn = tokens[:, i + 1]
        assert bool(((r[0].double() - lp.gather(1, drawn[:, None])[:, 0]).abs() <= 1e-5).all())
        assert bool(((r[1].double() + (lp.exp() * lp).sum(1)).abs() <= 1e-5).all())
        assert torch.equal(r[3].long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :3])
    # whole hypotheses at once, and from the middle on
    at_once, _ = binding.tdt_paged_attn(q, cache, table, lens, lens)
    assert bool(((at_once.double() - out).abs() <= bound).all())
    tail, _ = binding.tdt_paged_attn(q[:, 20:], cache, table, lens)
    assert bool(((tail.double() - out[:, 20:]).abs() <= bound[:, 20:]).all())


def test_on_two_streams_with_workspaces_of_their_own(binding):
    """Two utterances' calls on two streams at once give what they give one after the other."""
    embed, vocab, uniforms = _projections(5)
    runs = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache = binding.PagedCache.empty(80, 16, K, D, E4M3)
        table = torch.randperm(80, generator=g, device="cuda").view(1, 80).to(torch.int32)
        tokens = torch.randint(0, VOCAB, (1, 1200), generator=g, device="cuda")
        runs.append((cache, table, _heads(embed, tokens), i64([1200])))

    def call(cache, table, heads, lens):
        binding.tdt_cache_write(heads[1], heads[2], cache, table, lens)
        return binding.tdt_paged_attn(heads[0], cache, table, lens, need_lse=True)

    want = [call(*r) for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(call(*r))
        torch.cuda.synchronize()
        for w, x in zip(want, got):
            assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
