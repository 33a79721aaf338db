"""A hybrid transducer / attention decoder on the library's operators, with random weights.

Training: one step of the TDT loss on joint outputs together with an attention decoder whose label states
read each other causally, and the encoder's frames around the place where the transducer emits each label;
its loss is the labels' negative log-probability (tdt_loss, cross_attention, token_logprobs, all
differentiable).  Decoding: the attention decoder extends a beam of hypotheses token by token; each step
writes the new label states' keys and values into a paged cache, quantised, reads the cache and the
frames, draws a token for each hypothesis and takes its log-probability (tdt_cache_write, tdt_paged_attn,
tdt_cross_attn_fwd, tdt_sample, tdt_token_logprobs_fwd).  Rescoring: whole hypotheses read the same cache at
once.

    python examples/attention_decoder.py [--frames 200] [--labels 40] [--vocab 8193] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from transducer_loss_asr_gb300 import binding  # noqa: E402
from transducer_loss_asr_gb300.autograd import cross_attention, tdt_loss, token_logprobs  # noqa: E402

DURATIONS = [0, 1, 2, 3, 4]


class AttentionDecoder(torch.nn.Module):
    """Label states -> causal attention to each other -> cross attention over the frames -> token logits."""

    def __init__(self, vocab: int, width: int, heads: int, key_heads: int, head_dim: int):
        super().__init__()
        self.heads, self.key_heads, self.head_dim = heads, key_heads, head_dim
        self.embed = torch.nn.Embedding(vocab, width)
        self.to_qkv = torch.nn.Linear(width, (heads + 2 * key_heads) * head_dim, bias=False)
        self.to_state = torch.nn.Linear(heads * head_dim, width, bias=False)
        self.to_q = torch.nn.Linear(width, heads * head_dim, bias=False)
        self.to_kv = torch.nn.Linear(width, 2 * key_heads * head_dim, bias=False)
        self.to_out = torch.nn.Linear(heads * head_dim, width, bias=False)
        self.to_vocab = torch.nn.Linear(width, vocab, bias=False)

    def keys_values(self, frames):
        """k, v [B, T, key_heads, head_dim]: slices of one projection, no copies."""
        kv = self.to_kv(frames).unflatten(-1, (2, self.key_heads, self.head_dim))
        return kv[:, :, 0], kv[:, :, 1]

    def label_heads(self, tokens):
        """Embeddings, and q, k, v of the label states: slices of one projection."""
        x = self.embed(tokens)
        qkv = self.to_qkv(x).unflatten(-1, (self.heads + 2 * self.key_heads, self.head_dim))
        H, K = self.heads, self.key_heads
        return x, qkv[:, :, :H], qkv[:, :, H:H + K], qkv[:, :, H + K:]

    def queries(self, x, read):
        """Queries to the frames, from embeddings and what the label states read of each other."""
        return self.to_q(x + self.to_state(read.flatten(2))).unflatten(-1, (self.heads, self.head_dim))

    def logits(self, read):
        return self.to_vocab(self.to_out(read.flatten(2)))

    def forward(self, tokens, k, v, frame_lens, label_lens, windows):
        x, q, lk, lv = self.label_heads(tokens)
        at = torch.arange(tokens.shape[1], dtype=torch.int32, device=tokens.device)
        causal = torch.stack([torch.zeros_like(at), at + 1], -1).expand(tokens.shape[0], -1, -1).contiguous()
        own = cross_attention(q, lk, lv, label_lens, label_lens, causal)
        return self.logits(cross_attention(self.queries(x, own), k, v, frame_lens, label_lens, windows))


def emission_windows(joint, frame_lens, blank, reach):
    """[B, U, 2]: `reach` frames to either side of where the transducer emits each label; the whole
    utterance for labels that the greedy walk does not reach."""
    _, _, at, _ = binding.tdt_greedy_decode(joint, frame_lens, DURATIONS, blank)
    at = at[:, :-1]
    whole = torch.stack([torch.zeros_like(at), torch.full_like(at, joint.shape[1])], -1)
    near = torch.stack([at - reach, at + reach + 1], -1)
    return torch.where((at >= 0)[..., None], near, whole).contiguous()


def train_step(model, frames, frame_lens, labels, label_lens, joint, blank, reach=64):
    """TDT loss + the labels' mean negative log-probability under the attention decoder; returns both.  Gradients end up in the model and in joint.grad."""
    transducer = tdt_loss(joint, labels, frame_lens, label_lens, DURATIONS, blank)
    tokens = labels.clamp_min(0)
    windows = emission_windows(joint.detach(), frame_lens, blank, reach)
    k, v = model.keys_values(frames)
    # label u reads the frames near label u + 1, which it predicts
    logits = model(tokens[:, :-1], k, v, frame_lens, label_lens - 1, windows[:, 1:].contiguous())
    logprobs = token_logprobs(logits, labels[:, 1:])[0]  # padded labels: 0
    attention = -logprobs.sum() / (label_lens - 1).sum()
    (transducer + attention).backward()
    return transducer.detach(), attention.detach()


@torch.no_grad()
def decode(model, frames, frame_lens, beam, steps, blank, generator, temperature=0.8, top_k=50, top_p=0.95, page=16):
    """Draws `beam` hypotheses for each utterance: (tokens [B, beam, steps], log-probabilities [B, beam] of the model,
    those of the hypotheses scored again at once)."""
    B, dev, N = frames.shape[0], frames.device, frames.shape[0] * beam
    k, v = model.keys_values(frames)
    # a hypothesis has pages of its own, in the order of their numbers here
    pages = (steps + page - 1) // page
    cache = binding.PagedCache.empty(N * pages, page, model.key_heads, model.head_dim, binding.E4M3, dev)
    table = torch.arange(N * pages, dtype=torch.int32, device=dev).view(N, pages)
    lens = torch.zeros(N, dtype=torch.int64, device=dev)
    tokens = torch.full((N, 1), blank, dtype=torch.long, device=dev)
    out, score = [tokens], torch.zeros(N, device=dev)

    def read(q):
        return binding.tdt_cross_attn_fwd(q, k, v, k_lens=frame_lens, need_lse=False)[0]

    for _ in range(steps):
        lens += 1
        x, q, lk, lv = model.label_heads(tokens)
        binding.tdt_cache_write(lk, lv, cache, table, lens)
        own, _ = binding.tdt_paged_attn(q, cache, table, lens)
        logits = model.logits(read(model.queries(x, own).view(B, beam, model.heads, model.head_dim))).flatten(0, 1)
        u = torch.rand(N, generator=generator, device=dev)
        tokens = binding.tdt_sample(logits, u, temperature, top_k, top_p)[0].long()
        score += binding.tdt_token_logprobs_fwd(logits, tokens).logprobs
        tokens = tokens.view(N, 1)
        out.append(tokens)
    tokens = torch.cat(out, 1)  # [N, 1 + steps], the first the start
    x, q, _, _ = model.label_heads(tokens[:, :-1])
    own, _ = binding.tdt_paged_attn(q, cache, table, lens, lens)
    states = model.queries(x, own).view(B, beam * steps, model.heads, model.head_dim)
    logits = model.logits(read(states)).flatten(0, 1)
    again = binding.tdt_token_logprobs_fwd(logits, tokens[:, 1:].flatten()).logprobs.view(B, beam, steps).sum(-1)
    return tokens[:, 1:].view(B, beam, steps), score.view(B, beam), again


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 4), ("frames", 200), ("labels", 40), ("vocab", 8193), ("width", 512), ("heads", 8),
                        ("key-heads", 8), ("head-dim", 64), ("beam", 4), ("steps", 20), ("seed", 1)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    dev, dtype = torch.device("cuda"), torch.bfloat16
    torch.manual_seed(a.seed)
    g = torch.Generator(device=dev).manual_seed(a.seed)
    blank = a.vocab - 1
    model = AttentionDecoder(a.vocab, a.width, a.heads, a.key_heads, a.head_dim).to(dev, dtype)
    frames = torch.randn(a.batch, a.frames, a.width, generator=g, device=dev).to(dtype)
    frame_lens = torch.randint((a.frames + 1) // 2, a.frames + 1, (a.batch,), generator=g, device=dev)
    label_lens = torch.randint((a.labels + 1) // 2, a.labels + 1, (a.batch,), generator=g, device=dev)
    labels = torch.randint(0, blank, (a.batch, a.labels), generator=g, device=dev)
    labels = labels.masked_fill(torch.arange(a.labels, device=dev) >= label_lens[:, None], -100)
    joint = torch.randn(a.batch, a.frames, a.labels + 1, a.vocab + len(DURATIONS), generator=g, device=dev).to(dtype)
    joint.requires_grad_(True)
    transducer, attention = train_step(model, frames, frame_lens, labels, label_lens, joint, blank)
    tokens, score, again = decode(model, frames, frame_lens, a.beam, a.steps, blank, g)
    print("transducer loss %.4f, attention loss %.4f" % (transducer.item(), attention.item()))
    print("%d hypotheses of %d tokens for each of %d utterances; mean log-probability %.3f, scored at once %.3f"
          % (a.beam, a.steps, a.batch, score.mean().item(), again.mean().item()))
    return model, joint, tokens, score


if __name__ == "__main__":
    main()
