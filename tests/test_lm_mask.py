"""Rows that the vocabulary cross entropy ignores: nothing they hold reaches the
gradients, for every kernel that makes them."""

import pytest
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D,gap", [(70, 900, 96, 0), (70, 900, 64, 3), (300, 2000, 128, 0), (70, 900, 256, 0),
                                       (300, 2000, 200, 1)])
@pytest.mark.parametrize("size", [1.0, 1e10])
@pytest.mark.parametrize("what", [3e38, float("inf"), float("nan")])
def test_ignored_rows_of_any_values(n, V, D, gap, t, size, what):
    # 3e38 is finite, but its logits are not
    h, w, target, grad = ops.xent_inputs(n, V, D, t, gap, n + D)
    h, w = (h.double() / size).to(t), (w.double() * size).to(t)
    ignored = torch.arange(n, device=ops.DEV) % 7 == 3
    target[ignored] = -100
    clean = h.clone()
    clean[ignored] = 0
    x = tt.VocabCrossEntropy(V, D)
    ref = x.loss_and_grad(clean, w, target, grad)
    for cols in (slice(0, 1), slice(None)):
        h[ignored, cols] = what
        if cols == slice(None):
            h[ignored, 1::2] = -what
        got = x.loss_and_grad(h, w, target, grad)
        assert (got[0][ignored] == 0).all() and (got[2][ignored] == 0).all()
        assert all(torch.equal(p[~ignored], q[~ignored]) for p, q in zip(got[:3], ref[:3]))
        assert torch.equal(got[3], ref[3])
        assert torch.isfinite(got[2]).all() and torch.isfinite(got[3]).all()
        # the row's own lse is its logits', as forward says
        assert torch.equal(got[1].nan_to_num(7.0), x.forward(h, w, target)[1].nan_to_num(7.0))
    assert x.poll_error() == 0
