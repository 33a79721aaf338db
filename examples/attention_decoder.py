"""A hybrid transducer / attention decoder on the library's operators, with random weights.

Training: one step of the TDT loss on joint outputs together with an attention decoder whose label states
read the encoder's frames around the place where the transducer emits each label (tdt_loss,
cross_attention, both differentiable).  Decoding: the attention decoder extends a beam of hypotheses
token by token, every step one cross attention of a few rows to the frames and one draw of a token for
each hypothesis (tdt_cross_attn_fwd, tdt_sample).

    python examples/attention_decoder.py [--frames 200] [--labels 40] [--vocab 8193] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from transducer_loss_asr_gb300 import binding  # noqa: E402
from transducer_loss_asr_gb300.autograd import cross_attention, tdt_loss  # noqa: E402

DURATIONS = [0, 1, 2, 3, 4]


class AttentionDecoder(torch.nn.Module):
    """Label states -> cross attention over the frames -> token logits."""

    def __init__(self, vocab: int, width: int, heads: int, key_heads: int, head_dim: int):
        super().__init__()
        self.heads, self.key_heads, self.head_dim = heads, key_heads, head_dim
        self.embed = torch.nn.Embedding(vocab, width)
        self.to_q = torch.nn.Linear(width, heads * head_dim, bias=False)
        self.to_kv = torch.nn.Linear(width, 2 * key_heads * head_dim, bias=False)
        self.to_out = torch.nn.Linear(heads * head_dim, width, bias=False)
        self.to_vocab = torch.nn.Linear(width, vocab, bias=False)

    def keys_values(self, frames):
        """k, v [B, T, key_heads, head_dim]: slices of one projection, no copies."""
        kv = self.to_kv(frames).unflatten(-1, (2, self.key_heads, self.head_dim))
        return kv[:, :, 0], kv[:, :, 1]

    def queries(self, tokens):
        return self.to_q(self.embed(tokens)).unflatten(-1, (self.heads, self.head_dim))

    def forward(self, tokens, k, v, frame_lens, label_lens, windows):
        read = cross_attention(self.queries(tokens), k, v, frame_lens, label_lens, windows)
        return self.to_vocab(self.to_out(read.flatten(2)))


def emission_windows(joint, frame_lens, blank, reach):
    """[B, U, 2]: `reach` frames to either side of where the transducer emits each label; the whole
    utterance for labels that the greedy walk does not reach."""
    _, _, at, _ = binding.tdt_greedy_decode(joint, frame_lens, DURATIONS, blank)
    at = at[:, :-1]
    whole = torch.stack([torch.zeros_like(at), torch.full_like(at, joint.shape[1])], -1)
    near = torch.stack([at - reach, at + reach + 1], -1)
    return torch.where((at >= 0)[..., None], near, whole).contiguous()


def train_step(model, frames, frame_lens, labels, label_lens, joint, blank, reach=64):
    """TDT loss + attention cross entropy; returns both.  Gradients end up in the model and in joint.grad."""
    transducer = tdt_loss(joint, labels, frame_lens, label_lens, DURATIONS, blank)
    tokens = labels.clamp_min(0)
    windows = emission_windows(joint.detach(), frame_lens, blank, reach)
    k, v = model.keys_values(frames)
    # label u reads the frames near label u + 1, which it predicts
    logits = model(tokens[:, :-1], k, v, frame_lens, label_lens - 1, windows[:, 1:].contiguous())
    attention = torch.nn.functional.cross_entropy(logits.flatten(0, 1).float(), labels[:, 1:].flatten(),
                                                  ignore_index=-100)
    (transducer + attention).backward()
    return transducer.detach(), attention.detach()


@torch.no_grad()
def decode(model, frames, frame_lens, beam, steps, blank, generator, temperature=0.8, top_k=50, top_p=0.95):
    """Draws `beam` hypotheses for each utterance: (tokens [B, beam, steps], log-probabilities [B, beam])."""
    B = frames.shape[0]
    k, v = model.keys_values(frames)
    tokens = torch.full((B, beam), blank, dtype=torch.long, device=frames.device)
    out, score = [], torch.zeros(B, beam, device=frames.device)
    for _ in range(steps):
        read, _ = binding.tdt_cross_attn_fwd(model.queries(tokens), k, v, k_lens=frame_lens, need_lse=False)
        logits = model.to_vocab(model.to_out(read.flatten(2))).flatten(0, 1)
        u = torch.rand(B * beam, generator=generator, device=frames.device)
        drawn, logp = binding.tdt_sample(logits, u, temperature, top_k, top_p)
        tokens = drawn.view(B, beam).long()
        out.append(tokens)
        score += logp.view(B, beam)
    return torch.stack(out, -1), score


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
    tokens, score = decode(model, frames, frame_lens, a.beam, a.steps, blank, g)
    print("transducer loss %.4f, attention loss %.4f" % (transducer.item(), attention.item()))
    print("%d hypotheses of %d tokens for each of %d utterances; mean log-probability %.3f"
          % (a.beam, a.steps, a.batch, score.mean().item()))
    return model, joint, tokens, score


if __name__ == "__main__":
    main()
