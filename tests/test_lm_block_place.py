"""The norms between blocks in place: a backward after them takes x and the
residual from before the call."""

import pytest
import test_lm_block as block
import torch

import tensor_train_compressed_gather_amd as tt

F32, BF16 = block.F32, block.BF16


@pytest.mark.gpu
@pytest.mark.parametrize("kind,post", [("rms", False), ("layer", True)])
@pytest.mark.parametrize("n,D", [(5, 513), (40, 1000), (3, 4100)])
def test_backward_of_a_forward_in_place(n, D, kind, post):
    x, res, kw, gy, gh = block.make(n, D, BF16, BF16, kind, post, "vector", F32, 0, 3)
    op = tt.BlockNorm(D, kind=kind, post=post)
    y, h, stats = op.forward(x, res, **kw)
    back = {k: kw[k] for k in ("gate", "gamma", "post_gamma", "post_beta")}
    want = op.backward(gy, gh, x, res, stats, **back)
    x2, res2 = x.clone(), res.clone()
    y2, h2, stats2 = op.forward(x2, res2, out=x2, out_h=res2, **kw)
    assert y2 is x2 and h2 is res2 and torch.equal(y2, y) and torch.equal(h2, h) and torch.equal(stats2, stats)
    got = op.backward(gy, gh, x, res, stats2, **back)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))
