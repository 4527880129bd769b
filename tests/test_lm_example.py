"""The example model: the TT table, the lookup, the norm, the loss and AdamW in
one training step, on the GPU; its gradients against autograd in 64 bits."""

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("next_token", os.path.join(ROOT, "examples", "next_token.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_the_example_learns(bits):
    first, last = example().train(150, bits, B=2048)
    # from about log(1000) = 6.9 towards the noise's entropy, about 1
    assert first > 6.0 and last < 0.6 * first


def test_the_example_takes_the_gradient_of_its_loss():
    ex = example()
    model = ex.NextToken()
    context, target = next(ex.batches(model, 64))
    before = [p.clone() for p in model.params]
    grads = []
    model.opt.step = lambda gs: grads.extend(gs)
    loss = model.step(context, target)
    model.check()
    assert all(torch.equal(p, q) for p, q in zip(before, model.params))

    # the same model in 64 bits: rows of the TT table by the chain of its cores
    leaves = [p.double().requires_grad_() for p in before]
    (c0, c1, c2), weight, gamma, beta = leaves[:3], *leaves[3:]
    t = context.reshape(-1)
    i0, i1, i2 = t // 100, t // 10 % 10, t % 10
    rows = torch.einsum("nap,npbq,nqc->nabc", c0[i0][:, 0], c1[i1], c2[i2][..., 0]).reshape(len(t), -1)
    x = rows.view(64, -1, model.D).sum(1) + math.sqrt(model.D) * weight[context[:, -1]]
    y = torch.nn.functional.layer_norm(x, (model.D,), gamma, beta, 1e-5)
    ref = torch.nn.functional.cross_entropy(y @ weight.t(), target, ignore_index=ex.IGNORE, reduction="none")
    counts = (target != ex.IGNORE).sum()
    (ref.sum() / counts).backward()
    # fp32 sums of up to 64 x 1000 terms, each to 2^-22: far below 1e-4 of the largest value
    assert float((loss.double() - ref.detach()).abs().max()) <= 1e-4
    for g, leaf in zip(grads, leaves):
        assert float((g.double() - leaf.grad).abs().max()) <= 1e-4 * float(leaf.grad.abs().max())
