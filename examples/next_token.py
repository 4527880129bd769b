"""A small next-token model around a tensor-train table, trained end to end.

The tokens of the context are pooled from a TT-compressed table, the last
token's row comes from a dense table that the output layer shares; their sum
is normalised and scored against the whole vocabulary:

    x = pool(TT table, context) + sqrt(D) W[last]      TTEmbeddingBag, TokenEmbedding
    y = layer norm(x)                                  LayerNorm
    loss = cross entropy(y W^T, next)                  VocabCrossEntropy

The gradients take the same way back (the dense table's two are added up in
place) and one AdamW step updates the TT cores, the dense table and the norm.
Tokens are synthetic: each follows its predecessor by a fixed table, with noise.

    python examples/next_token.py [--steps 200] [--bits 8]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_train_compressed_gather_amd as tt  # noqa: E402
from tensor_train_compressed_gather_amd.workloads import Table  # noqa: E402

IGNORE = -100


class NextToken:
    def __init__(self, device="cuda", context: int = 4, rank: int = 16, state_bits: int = 32, lr: float = 5e-3,
                 seed: int = 0):
        self.table = Table(1000, (10, 10, 10), (4, 4, 4), (1, rank, rank, 1), 0.1, "uniform")
        self.V, self.D, self.context, self.device = self.table.N, self.table.D, context, device
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(shape, std):
            return torch.empty(shape, device=device).normal_(0.0, std, generator=g)

        self.cores = [normal(s, 0.3) for s in self.table.core_shapes()]
        self.weight = normal((self.V, self.D), 1.0 / math.sqrt(self.D))
        self.gamma, self.beta = torch.ones(self.D, device=device), torch.zeros(self.D, device=device)
        self.bag = tt.TTEmbeddingBag([self.table], device)
        self.last = tt.TokenEmbedding(self.V, self.D, scale=math.sqrt(self.D), device=device)
        self.norm = tt.LayerNorm(self.D, device=device)
        self.loss = tt.VocabCrossEntropy(self.V, self.D, ignore_index=IGNORE, device=device)
        self.params = [*self.cores, self.weight, self.gamma, self.beta]
        self.opt = tt.AdamW(self.params, lr=lr, state_bits=state_bits, seed=seed)

    def step(self, context, target):
        """One training step on context tokens [B][context] and their next
        tokens [B] (IGNORE: not counted); returns the losses [B]."""
        B = target.shape[0]
        tokens = context.reshape(-1)
        offsets = torch.arange(0, B * self.context + 1, self.context, device=self.device)
        last = context[:, -1].contiguous()
        x = self.bag.forward(self.cores, tokens, offsets, B) + self.last.forward(self.weight, last)
        y, mean, rstd = self.norm.forward(x, self.gamma, self.beta)
        counts = target != IGNORE
        grad_loss = counts / counts.sum().clamp(min=1)
        loss, _, dy, dweight = self.loss.loss_and_grad(y, self.weight, target, grad_loss)
        dx, dgamma, dbeta = self.norm.backward(dy, x, self.gamma, mean, rstd)
        dcores = self.bag.backward(dx, self.cores, tokens, offsets, B, flags=tt.TT_EMB_REUSE_GROUPING)
        self.last.backward(dx, last, grad_weight=dweight, accumulate=True)
        self.opt.step([*dcores, dweight, dgamma, dbeta])
        return loss

    def check(self):
        """Raise if a call met a token out of range (synchronises)."""
        for op in (self.bag, self.last, self.loss):
            status = op.poll_error()
            if status:
                raise tt.TTEmbError(status, type(op).__name__)


def batches(model: NextToken, B: int, seed: int = 1):
    """Endless (context, target) pairs: nine times of ten the next token is
    the last one's successor in a fixed permutation, else any token; one
    target in sixteen is not counted."""
    g = torch.Generator(device=model.device)
    g.manual_seed(seed)
    follows = torch.randperm(model.V, device=model.device, generator=g)
    while True:
        context = torch.randint(0, model.V, (B, model.context), device=model.device, generator=g)
        target = follows[context[:, -1]]
        other = torch.randint(0, model.V, (B,), device=model.device, generator=g)
        u = torch.rand(B, device=model.device, generator=g)
        target = torch.where(u < 0.1, other, target)
        yield context, torch.where(u > 1 - 1 / 16, IGNORE, target)


def train(steps: int, state_bits: int = 32, B: int = 4096, report: int = 0):
    """Mean loss of the first and of the last step."""
    model = NextToken(state_bits=state_bits)
    first = last = None
    for i, (context, target) in zip(range(steps), batches(model, B)):
        loss = model.step(context, target)
        if i == 0 or i + 1 == steps or (report and i % report == 0):
            last = float(loss.sum() / (target != IGNORE).sum())
            first = last if i == 0 else first
            if report:
                print(f"step {i:5d}  loss {last:.4f}", flush=True)
    model.check()
    return first, last


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32, help="bits of the AdamW states")
    a = ap.parse_args()
    train(a.steps, a.bits, report=20)
