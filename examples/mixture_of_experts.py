"""A small mixture-of-experts language model, trained and sampled with the language-model
operators: route_tokens chooses each token's experts and gives their gate weights and the
balance loss, both differentiable; sample_tokens draws the next tokens.

  python examples/mixture_of_experts.py [--steps N] [--seed S]

The text is synthetic: sequences of a random walk over the vocabulary (the next token is the
last one plus 1, 2 or 3), some of them padded, so a model that learns gets from ln 64 = 4.16
to ln 3 = 1.10.  Needs a GPU.
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import sampling_threshold_filtering_amd as stf  # noqa: E402

VOCAB, WIDTH, EXPERTS, CHOSEN, LENGTH, BATCH = 64, 64, 8, 2, 48, 64


class Layer(torch.nn.Module):
    """CHOSEN of EXPERTS two-layer experts for each token."""

    def __init__(self):
        super().__init__()
        self.router = torch.nn.Linear(WIDTH, EXPERTS, bias=False)
        self.up = torch.nn.Parameter(torch.randn(EXPERTS, WIDTH, 2 * WIDTH) * WIDTH ** -0.5)
        self.down = torch.nn.Parameter(torch.randn(EXPERTS, 2 * WIDTH, WIDTH) * (2 * WIDTH) ** -0.5)

    def forward(self, x, mask=None):
        """x [tokens, WIDTH]; mask [tokens]: padding takes no part.  (output, Routing)"""
        r = stf.route_tokens(self.router(x), CHOSEN, normalize=True, mask=mask, balance=True)
        out = torch.zeros_like(x)
        for e in range(EXPERTS):
            token, slot = (r.experts == e).nonzero(as_tuple=True)
            y = torch.relu(x[token] @ self.up[e]) @ self.down[e]
            out = out.index_add(0, token, y * r.weights[token, slot].unsqueeze(1))
        return x + out, r


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(VOCAB, WIDTH)
        self.layers = torch.nn.ModuleList(Layer() for _ in range(2))
        self.head = torch.nn.Linear(WIDTH, VOCAB, bias=False)

    def forward(self, tokens, mask=None):
        x, routings = self.embed(tokens), []
        for layer in self.layers:
            x, r = layer(x, mask)
            routings.append(r)
        return self.head(x), routings


def text(gen):
    """(tokens, which of them are not padding)"""
    step = torch.randint(1, 4, (BATCH, LENGTH), generator=gen, device="cuda")
    length = torch.randint(LENGTH // 2, LENGTH + 1, (BATCH, 1), generator=gen, device="cuda")
    return step.cumsum(1) % VOCAB, torch.arange(LENGTH, device="cuda") < length


def main(steps: int = 150, seed: int = 0, quiet: bool = False):
    """(first loss, last loss, share of drawn tokens that the text allows)"""
    torch.manual_seed(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    model = Model().cuda()
    optimiser = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for i in range(steps):
        tokens, real = text(gen)
        mask = real[:, :-1].reshape(-1)
        logits, routings = model(tokens[:, :-1].reshape(-1), mask)
        loss = torch.nn.functional.cross_entropy(logits[mask], tokens[:, 1:].reshape(-1)[mask])
        balance = sum(r.loss for r in routings)
        optimiser.zero_grad()
        (loss + 0.01 * balance).backward()
        optimiser.step()
        losses.append(float(loss.detach()))
        if not quiet and i % 25 == 0:
            print(f"step {i:4d}  loss {losses[-1]:.3f}  balance {float(balance.detach()) / 2:.3f} (1: even)  "
                  f"first layer's counts {routings[0].counts.tolist()}", flush=True)
    with torch.no_grad():
        last = torch.randint(0, VOCAB, (BATCH,), generator=gen, device="cuda")
        lines, allowed = [last], 0
        for _ in range(20):
            logits, _ = model(last)
            u = torch.rand(BATCH, generator=gen, device="cuda")
            new, logprob = stf.sample_tokens(logits, u, temperature=0.8, top_k=8, top_p=0.95)
            step = (new - last) % VOCAB
            allowed += int(((step >= 1) & (step <= 3)).sum())
            last = new
            lines.append(new)
    if not quiet:
        print("a drawn line:", torch.stack(lines)[:, 0].tolist())
        print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; allowed by the text: {allowed / (20 * BATCH):.3f}")
    return losses[0], losses[-1], allowed / (20 * BATCH)


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=150)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args()
    main(a.steps, a.seed)
