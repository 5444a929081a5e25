"""A small fine-tuning run: layer norms, DoRA layers, token log probabilities and AdamW together.

    python examples/finetune.py [--steps 60] [--state-bits 8]

A frozen random network (embedding, two blocks of layer norm and a square projection with a residual,
a norm and a head) is given DoRA adapters and learns, through them alone, the successor of each token
in a fixed random order.  The first quarter of every sequence is prompt (no target).  Afterwards one
token at a time is scored and its likeliest alternatives printed, as a server would.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from parameter_efficient_fine_dora_amd.module import DoRALinear, LayerNorm, token_logprob  # noqa: E402
from parameter_efficient_fine_dora_amd.optim import AdamW  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab, width, rank, dtype, device="cuda"):
        super().__init__()

        def weight(rows, cols):
            return (torch.randn(rows, cols, device=device) / cols ** 0.5).to(dtype)

        self.register_buffer("table", torch.randn(vocab, width, device=device).to(dtype))
        self.norms = torch.nn.ModuleList(LayerNorm(width, device=device, dtype=dtype) for _ in range(3))
        self.mixes = torch.nn.ModuleList(DoRALinear(weight(width, width), r=rank) for _ in range(2))
        self.head = DoRALinear(weight(vocab, width), r=rank)

    def forward(self, tokens):
        h = self.table[tokens]
        for norm, mix in zip(self.norms, self.mixes):
            h = h + mix(norm(h))
        return self.head(self.norms[2](h))


def train(steps=60, state_bits=8, vocab=1000, width=256, rank=16, batch=16, length=64, seed=0,
          dtype=torch.bfloat16, lr=1e-2, report=print):
    torch.manual_seed(seed)
    model = Model(vocab, width, rank, dtype)
    successor = torch.randperm(vocab, device="cuda")
    decayed = [p for n, p in model.named_parameters() if n.endswith((".A", ".B"))]
    others = [p for n, p in model.named_parameters() if not n.endswith((".A", ".B"))]
    opt = AdamW([dict(params=decayed), dict(params=others, weight_decay=0.0)], lr=lr,
                state_bits=state_bits, master=True, max_norm=1.0)
    losses = []
    for step in range(steps):
        tokens = torch.randint(vocab, (batch, length), device="cuda")
        targets = successor[tokens]
        targets[:, :length // 4] = -100
        logp, entropy, _, _ = token_logprob(model(tokens), targets)
        count = batch * (length - length // 4)
        loss = -logp.sum() / count - 1e-3 * entropy.sum() / count
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report and (step % 10 == 0 or step == steps - 1):
            report(f"step {step:3d}  loss {float(loss.detach()):.3f}  gradient norm {float(opt.grad_norm):.3f}",
                   flush=True)
    return model, successor, [float(x) for x in losses]


@torch.no_grad()
def serve(model, successor, token, top=5):
    """Scores the successor of one token; returns (logp, entropy, [(alternative, logp)])."""
    t = torch.tensor([token], device="cuda")
    logp, entropy, best, index = token_logprob(model(t), successor[t], top=top)
    return float(logp), float(entropy), list(zip(index[0].tolist(), best[0].tolist()))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    model, successor, _ = train(a.steps, a.state_bits)
    for token in (3, 14, 159):
        logp, entropy, best = serve(model, successor, token)
        print(f"token {token} -> {int(successor[token])}: log p {logp:.2f}, entropy {entropy:.2f}, best",
              ", ".join(f"{i} ({lp:.2f})" for i, lp in best))


if __name__ == "__main__":
    main()
