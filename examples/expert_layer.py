"""Trains a small mixture-of-experts block on synthetic data, with the layer operators as a training
program uses them:

    python examples/expert_layer.py [--steps 40] [--gated] [--checkpoint int8]

Each token goes to the expert that its router scores highest.  A step is: RMS norm of the stream
(with the residual's addition), the tokens sorted by expert, two products grouped by expert with an
activation between them, and back.  The experts' weights are updated inside their layers' backward
pass; the gains, the router and the output head take one step over many tensors.  With --gated the
experts are gated blocks; --checkpoint keeps the activations for the backward pass in 8 bits.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import optimizer_step_weight_amd as forge  # noqa: E402
from optimizer_step_weight_amd.autograd import FusedExperts, FusedGatedExperts, RMSNorm  # noqa: E402


class ExpertBlock(torch.nn.Module):
    def __init__(self, width: int, hidden: int, experts: int, hyper, *, gated: bool = False, checkpoint=None):
        super().__init__()
        self.experts = experts
        self.norm_in, self.norm_out = RMSNorm(width, checkpoint=checkpoint), RMSNorm(width, checkpoint=checkpoint)
        self.router = torch.nn.Parameter(torch.randn(experts, width, device="cuda") * width ** -0.5)
        kw = dict(hyper=hyper, checkpoint=checkpoint)
        if gated:
            self.block = FusedGatedExperts(experts, width, hidden, seed=1, **kw)
        else:
            self.up = FusedExperts(experts, width, hidden, seed=1, **kw)
            self.down = FusedExperts(experts, hidden, width, seed=2, **kw)
            self.block = lambda y, ends: self.down(F.silu(self.up(y, ends)), ends)
        self.head = torch.nn.Parameter(torch.randn(width, width, device="cuda") * width ** -0.5)

    def forward(self, x):
        y = self.norm_in(x)
        score, expert = torch.softmax(y.float() @ self.router.t(), 1).max(1)
        order = torch.sort(expert, stable=True).indices
        ends = torch.bincount(expert, minlength=self.experts).cumsum(0).to(torch.int32)
        out = self.block(y[order], ends)
        back = torch.empty_like(out).index_copy(0, order, out) * score.unsqueeze(1).to(out.dtype)
        y, _ = self.norm_out(back, residual=x)
        return y.float() @ self.head.t()


def train(steps: int, *, tokens: int = 1024, width: int = 256, hidden: int = 512, experts: int = 8, lr: float = 2e-3,
          gated: bool = False, checkpoint=None):
    """Losses of a fit to a random teacher."""
    torch.manual_seed(0)
    hyper = {"lr": lr}
    block = ExpertBlock(width, hidden, experts, hyper, gated=gated, checkpoint=checkpoint)
    params = [p for p in block.parameters() if p.numel()]
    for p in params:
        p.grad = torch.zeros_like(p)      # the plan holds these; backward adds to them
    moments = [[torch.zeros_like(p) for p in params] for _ in range(2)]
    plan = forge.MultiStep([p.data for p in params], [p.grad for p in params], *moments, opt="adamw")
    teacher = torch.randn(width, width, device="cuda") * width ** -0.5
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, width, device="cuda").to(torch.bfloat16)
        loss = F.mse_loss(block(x), torch.tanh(x.float() @ teacher))
        for p in params:
            p.grad.zero_()
        loss.backward()
        plan.step(step=step, hyper=hyper)
        losses.append(loss.detach())
    return [float(t) for t in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--gated", action="store_true")
    ap.add_argument("--checkpoint", choices=["int8", "fp8"])
    args = ap.parse_args()
    for i, loss in enumerate(train(args.steps, gated=args.gated, checkpoint=args.checkpoint)):
        if i % 5 == 0:
            print(f"step {i + 1}: loss {loss:.4f}", flush=True)
