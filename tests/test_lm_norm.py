"""Statistics of layer norm rows that hold NaN or infinities."""

import pytest
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("t", ops.TYPES)
@pytest.mark.parametrize("D", [3, 96, 100, 1024, 5000, 16384])
def test_statistics_of_rows_that_are_not_finite(D, t):
    n = 9
    x = ops.rows(ops.gen(D), n, D, t).clone()
    op = tt.LayerNorm(D)
    clean = op.forward(x)
    x[1, D // 2], x[3, 0], x[4, D - 1] = NAN, INF, -INF
    x[6, 0], x[6, 1] = INF, -INF
    y, mean, rstd = op.forward(x)
    bad = torch.tensor([1, 3, 4, 6], device=ops.DEV)
    good = torch.tensor([0, 2, 5, 7, 8], device=ops.DEV)
    assert rstd[bad].isnan().all() and y[bad].isnan().all()
    assert mean[1].isnan() and mean[3] == INF and mean[4] == -INF and mean[6].isnan()
    for got, ref in zip((y, mean, rstd), clean):
        assert torch.equal(got[good], ref[good])
    dy = ops.rows(ops.gen(1), n, D, t)
    dx = op.backward(dy, x, None, mean, rstd)[0]
    assert dx[bad].isnan().all() and torch.isfinite(dx[good]).all()
