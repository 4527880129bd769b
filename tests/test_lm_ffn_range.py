"""The gated feed-forward block's activations and their slopes over the whole
range of the gate, in each type.

One row, D = 1: with the gate's values z in `pre` and `up` for the other
projection's, w_out 1 and grad_y `gy`, the gradient of w_in is the slopes times up
gy and the values times gy, and that of w_out the values times up gy, each a sum of
one term.  (Powers of two lift what fp16 would round to a multiple of 2^-24.)"""

import pytest
import test_lm_ffn as ffn
import torch

import tensor_train_compressed_gather_amd as tt

DEV, U32 = ffn.DEV, ffn.U32


def derivatives(kind, t, z, up=1.0, gy=1.0):
    """Slopes, values (as p's gradient) and values (as a) of fp32 z."""
    F = z.numel()
    one = torch.ones((1, 1), device=DEV, dtype=t)
    op = tt.GatedFeedForward(1, F, activation=kind)
    pre = torch.cat([z, torch.full_like(z, up)])[None]
    _, dw_in, dw_out = op.backward(one * gy, one, pre, torch.ones((2 * F, 1), device=DEV, dtype=t),
                                   torch.ones((1, F), device=DEV, dtype=t))
    return dw_in[:F, 0].double() / up / gy, dw_in[F:, 0].double() / gy, dw_out[0].double() / up / gy


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


@pytest.mark.gpu
@pytest.mark.parametrize("t", [ffn.F32, ffn.BF16, ffn.F16])
@pytest.mark.parametrize("kind", ffn.ACTS)
def test_activations_keep_their_bits_in_the_tail(kind, t):
    # relative to the value: 16 bits u and what the exponential's argument of up to 122 is rounded to, 2^-15;
    # fp32 some 64 x 2^-24 (1 + z^2 / 2), as the argument z^2 / 2 is.  The slope is s + z s' with s = value / z
    F = 600
    z = torch.linspace(-12.9, 12.9, 2 * F, device=DEV)[:F] if kind == "gelu" else torch.linspace(-60, 60, F, device=DEV)
    if kind == "gelu_tanh":
        z = z / 10
    slope, value = reference(kind, z)
    s = (value / z.double()).abs()
    rel = 64 * U32 * (1 + z.double() ** 2) if t == ffn.F32 else ffn.ops.u(t) + 2.0 ** -14
    # (fp16 also rounds to a multiple of 2^-24, lifted or not)
    for up, gy in ((1.0, 1.0), (1024.0, 1.0), (1.0, 1024.0)) if t == ffn.F16 else ((1.0, 1.0),):
        got = derivatives(kind, t, z, up, gy)
        for x, ref, size, lift in ((got[0], slope, slope.abs() + 2 * s, up * gy), (got[1], value, value.abs(), gy),
                                   (got[2], value, value.abs(), up)):
            # (fp32's three terms lose the last bits of what is below 2^-100)
            tiny = {ffn.F16: 2.0 ** -24 / lift, ffn.BF16: 2.0 ** -120, ffn.F32: 2.0 ** -100}[t]
            assert ((x - ref).abs() <= rel * size + tiny).all(), (up, gy)
