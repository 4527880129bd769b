"""The gated feed-forward block's activations and their slopes over the whole
range of the gate, in each type.

One row, D = 1: with the gate's values z in `pre` and the other projection's 1,
grad_y and w_out 1, the gradient of w_in is the slopes and the values, and
that of w_out the values again, each a sum of one term."""

import pytest
import test_lm_ffn as ffn
import torch

import tensor_train_compressed_gather_amd as tt

DEV, U32 = ffn.DEV, ffn.U32


def derivatives(kind, t, z):
    """Slopes, values (as p's gradient) and values (as a) of fp32 z."""
    F = z.numel()
    one = torch.ones((1, 1), device=DEV, dtype=t)
    op = tt.GatedFeedForward(1, F, activation=kind)
    pre = torch.cat([z, torch.ones_like(z)])[None]
    _, dw_in, dw_out = op.backward(one, one, pre, torch.ones((2 * F, 1), device=DEV, dtype=t),
                                   torch.ones((1, F), device=DEV, dtype=t))
    return dw_in[:F, 0].double(), dw_in[F:, 0].double(), dw_out[0].double()


def reference(kind, z):
    leaf = z.double().requires_grad_()
    value = ffn.act64(kind, leaf)
    slope, = torch.autograd.grad(value.sum(), leaf)
    return slope, value.detach()


@pytest.mark.gpu
@pytest.mark.parametrize("t", [ffn.F32, ffn.BF16, ffn.F16])
@pytest.mark.parametrize("kind", ffn.ACTS)
def test_activations_of_large_values(kind, t):
    # slopes of 1 and 0, values of z and 0; silu's tail at -50 is 1e-20, its exponential off by 2^-24 of its
    # argument of 72 in 16 bits
    z = torch.logspace(1.7, 38.4, 221, device=DEV).float()
    z = torch.cat([z, -z, torch.tensor([1.1e13, 1.3e13, 1e14, 1.9e19, 1e20, -1e14, -1e20], device=DEV)])
    slope, value = reference(kind, z)
    rel = 128 * U32 if t == ffn.F32 else ffn.ops.u(t) + 2.0 ** -14
    tiny = 2.0 ** -24 if t == ffn.F16 else 1e-37
    got = derivatives(kind, t, z)
    fits = value.abs() <= torch.finfo(t).max
    assert fits.sum() > 20 and (got[0] == got[0]).all()
    for x, ref in ((got[0], slope), (got[1][fits], value[fits]), (got[2][fits], value[fits])):
        assert ((x - ref).abs() <= rel * ref.abs() + tiny).all()
