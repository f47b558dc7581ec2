"""A small language model trained and decoded with the library's operators around the head.

    python examples/train_and_decode.py [--steps N]

Training: one residual block whose gated, normalised output and the head's pre-norm are one
``block_norm``, the fused linear cross-entropy of the head, and ``clip_grad_norm_`` before the
optimizer's step. Decoding: the same block and head for single tokens, ``beam_select`` over beams and
vocabulary, ``beam_reorder`` of the recurrent state and the tokens so far. The task is to go on
with number sequences ``t' = (a t + b) mod V`` whose (a, b) shows in the first two tokens.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_cross_entropy_tcgen05_gb300 as flce  # noqa: E402

VOCAB, DIM, LENGTH = 256, 256, 16
RULES = [(1, 1), (1, 7), (5, 3), (3, 0)]


def sequences(n: int, generator, device):
    """n sequences of LENGTH + 1 tokens, each after one of the rules."""
    rule = torch.tensor(RULES, device=device)[torch.randint(len(RULES), (n,), generator=generator, device=device)]
    t = [torch.randint(VOCAB, (n,), generator=generator, device=device)]
    for _ in range(LENGTH):
        t.append((rule[:, 0] * t[-1] + rule[:, 1]) % VOCAB)
    return torch.stack(t, 1)


class Model(torch.nn.Module):
    """Embeddings of the last two tokens, one gated residual block, a head."""

    def __init__(self, device):
        super().__init__()
        kw = dict(device=device, dtype=torch.bfloat16)
        par = lambda *s: torch.nn.Parameter(torch.randn(*s, **kw) * s[-1] ** -0.5)  # noqa: E731
        self.last, self.before = par(VOCAB, DIM), par(VOCAB, DIM)
        self.up, self.down, self.head = par(4 * DIM, DIM), par(DIM, 4 * DIM), par(VOCAB, DIM)
        self.norm = flce.BlockNorm(DIM, post_norm=True, gate_init=1.0, gate_activation="tanh", **kw)

    def hidden(self, last, before):
        """Head inputs [N, DIM] for the last token and the embedding of the one before it."""
        residual = self.last[last] + before
        x = torch.nn.functional.gelu(residual @ self.up.t()) @ self.down.t()
        return self.norm(x, residual)[1]

    def loss(self, tokens):
        """Mean cross-entropy of every token from the third on."""
        before, last, target = tokens[:, :-2], tokens[:, 1:-1], tokens[:, 2:]
        y = self.hidden(last.reshape(-1), self.before[before.reshape(-1)])
        return flce.linear_cross_entropy(y, self.head, target.reshape(-1).int(), weight_layout="vd")


def train(model, steps: int, generator, max_norm: float = 1.0):
    """Losses and gradient norms of the steps."""
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    losses, norms = [], []
    for _ in range(steps):
        loss = model.loss(sequences(256, generator, model.head.device))
        opt.zero_grad()
        loss.backward()
        norms.append(flce.clip_grad_norm_(model.parameters(), max_norm))
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses), torch.stack(norms)


@torch.no_grad()
def decode(model, prompt, beams: int, length: int):
    """Beam search from two-token prompts [B, 2]: tokens [B, beams, 2 + length] and scores."""
    B, K, dev = prompt.shape[0], beams, prompt.device
    history = torch.zeros(B * K, 2 + length, dtype=torch.int32, device=dev)
    history[:, :2] = prompt.repeat_interleave(K, 0)
    last = history[:, 1].long()
    state = model.before[history[:, 0].long()]  # what a step keeps of the tokens before its last
    scores = torch.full((B, K), float("-inf"), device=dev)
    scores[:, 0] = 0.0  # at first the beams of a request are alike: one counts
    for i in range(length):
        logits = model.hidden(last, state) @ model.head.t()
        scores, parents, tokens = flce.beam_select(logits.view(B, K, VOCAB), scores)
        state = model.before[last]
        flce.beam_reorder([state, history], parents)
        last = tokens.view(-1).long()
        history[:, 2 + i] = tokens.view(-1)
    return history.view(B, K, -1), scores


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--beams", type=int, default=4)
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    model = Model("cuda")
    losses, norms = train(model, args.steps, g)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}, gradient norm {norms[0]:.3f} -> {norms[-1]:.3f}")
    tokens = sequences(6, g, "cuda")
    found, scores = decode(model, tokens[:, :2].int(), args.beams, 8)
    for want, got, s in zip(tokens.tolist(), found[:, 0].tolist(), scores[:, 0].tolist()):
        print(f"{want[:2]} -> {got[2:]} (wanted {want[2:10]}), log-probability {s:.3f}")
    return losses, norms, tokens, found, scores


if __name__ == "__main__":
    main()
