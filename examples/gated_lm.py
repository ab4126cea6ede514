"""A small recurrent language model on the gated linear scan: token embedding,
layers of input projection + gated scan, logits. It learns a synthetic language
(each token follows from the one two places before), with the layers' inputs
and pre-activations kept in 8 bits for the backward if asked, and then answers
token by token with the single-step form, its states in a pool.

    python examples/gated_lm.py [--steps 300] [--checkpoint int8]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import recurrent_networks_gb300 as rn  # noqa: E402

PAD = 0


class GatedLM:
    """V tokens, width E, `layers` scans of N heads of D channels."""

    def __init__(self, V=64, E=64, N=2, D=64, layers=2, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(device).requires_grad_(True)

        self.V, self.E, self.N, self.D = V, E, N, D
        self.embed = weight(V, E, scale=1 / math.sqrt(E))
        self.layers = []
        width = E
        for _ in range(layers):
            b = torch.zeros(4, N, D)
            b[1] = torch.linspace(0, 5, D)  # memories from one step to a hundred and fifty
            self.layers.append(dict(W=weight(4 * N * D, width, scale=1 / math.sqrt(width)),
                                    b=b.to(torch.bfloat16).to(device).requires_grad_(True)))
            width = N * D
        self.out = weight(V, width, scale=1 / math.sqrt(width))

    def parameters(self):
        return [self.embed] + [p for layer in self.layers for p in layer.values()] + [self.out]

    def forward(self, tokens, reset=None, lengths=None, checkpoint=None):
        """tokens [B,T] -> logits [B,T,V] and every layer's last state [B,1,N,D]."""
        B, T = tokens.shape
        x = rn.embedding(tokens, self.embed, scale=math.sqrt(self.E), padding_idx=PAD)
        states = []
        for layer in self.layers:
            Wx = rn.input_projection(x, layer["W"], checkpoint=checkpoint).reshape(B, T, 4, self.N, self.D)
            h, last = rn.gated_scan(Wx, layer["b"], function="linear", reset=reset, lengths=lengths,
                                    checkpoint=checkpoint)
            states.append(last)
            x = h.reshape(B, T, self.N * self.D)
        return rn.input_projection(x, self.out), states

    @torch.no_grad()
    def step(self, tokens, pools, slots):
        """One token of M running requests: tokens [M], pools per layer [P,N,D] (updated), slots [M]."""
        x = rn.embedding(tokens, self.embed, scale=math.sqrt(self.E))
        for layer, pool in zip(self.layers, pools):
            Wx = rn.input_projection(x, layer["W"]).reshape(-1, 4, self.N, self.D)
            x = rn.gated_scan_step(Wx, layer["b"], pool, slots).reshape(-1, self.N * self.D)
        return rn.input_projection(x, self.out)

    @torch.no_grad()
    def answer(self, prompts, lengths, count):
        """Greedy continuation of prompts [B,T] (row b has lengths[b] tokens) by `count` tokens."""
        B = prompts.shape[0]
        logits, states = self.forward(prompts, lengths=lengths)
        pools = [s[:, 0].contiguous() for s in states]
        slots = torch.arange(B, dtype=torch.int32, device=prompts.device)
        token = logits[torch.arange(B, device=prompts.device), lengths.long() - 1].float().argmax(-1)
        tokens = [token]
        for _ in range(count - 1):
            token = self.step(token, pools, slots).float().argmax(-1)
            tokens.append(token)
        return torch.stack(tokens, 1)


def language(B, T, V, seed, device="cuda"):
    """Sequences whose token follows from the one two places before."""
    g = torch.Generator().manual_seed(seed)
    t = torch.empty(B, T, dtype=torch.int64)
    t[:, :2] = torch.randint(1, V, (B, 2), generator=g)
    for k in range(2, T):
        t[:, k] = (t[:, k - 2] * 5 + 3) % (V - 1) + 1
    return t.to(device)


def train(model, steps=60, B=16, T=128, checkpoint=None, lr=3e-3):
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for k in range(steps):
        tokens = language(B, T + 1, model.V, seed=k)
        logits, _ = model.forward(tokens[:, :-1], checkpoint=checkpoint)
        loss = torch.nn.functional.cross_entropy(logits.float().reshape(-1, model.V), tokens[:, 1:].reshape(-1))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--checkpoint", choices=["int8"], default=None)
    a = ap.parse_args()
    model = GatedLM()
    losses = train(model, a.steps, checkpoint=a.checkpoint)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} after {a.steps} steps")
    seq = language(4, 48, model.V, seed=10_000)
    lengths = torch.tensor([32, 30, 24, 32], dtype=torch.int32, device="cuda")
    got = model.answer(seq[:, :32], lengths, 8)
    want = torch.stack([seq[b, n:n + 8] for b, n in enumerate(lengths.tolist())])
    print(f"{(got == want).float().mean().item():.0%} of the continuations' tokens are right")


if __name__ == "__main__":
    main()
