"""The vocabulary cross entropy with dL/dloss of very different size per row:
each row's gradient keeps its own precision."""

import pytest
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32 = ops.U32
SIZES = [(64, 500, 64, 0), (64, 500, 128, 3), (200, 3000, 100, 0), (64, 500, 256, 0), (300, 3000, 200, 1)]


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D,gap", SIZES)
@pytest.mark.parametrize("largest", [0, 60, -60])
def test_rows_keep_their_precision(n, V, D, gap, t, largest):
    h, w, target, _ = ops.xent_inputs(n, V, D, t, gap, n + D)
    grad = torch.exp2(torch.linspace(largest - 40, largest, n, device=ops.DEV))
    grad[1::2] *= -1.3
    grad[5], target[9] = 0.0, -100
    z, lse, loss, d, mag = ops.xent_reference(h, w, target, grad, -100)
    h64, w64 = h.double(), w.double()
    got = tt.VocabCrossEntropy(V, D).loss_and_grad(h, w, target, grad)
    ez = (6 * D + 8) * U32 * (h64.abs() @ w64.abs().t()).amax(1)
    # d's rounding (two fp16 terms: 2^-22, and 2^-38 of the row's gradient for small probabilities; or bf16's)
    size = (grad.double().abs() * (target != -100))[:, None]
    ed = ((ops.u(BF16) if t == BF16 else 2.0 ** -21) + 2 * ez + 220 * U32)[:, None] * mag + 2.0 ** -38 * size
    ref = d @ w64
    ops.close(got[2], ref, ed @ w64.abs() + 6 * (V + 8) * U32 * (mag @ w64.abs()) + ops.u(t) * ref.abs(), "dh")
    # two fp16 terms of a product that is scaled with the others: 2^-39 of the largest, of every row
    ref = d.t() @ h64
    floor = 2.0 ** -38 * (size * h64.abs()).amax() * (n + (mag / size.clamp(min=1e-300)).sum(0)[:, None])
    ops.close(got[3], ref, ed.t() @ h64.abs() + 6 * (n + 8) * U32 * (mag.t() @ h64.abs()) + ops.u(t) * ref.abs()
              + floor, "dw")
    assert (got[2][5] == 0).all() and (got[2][9] == 0).all()


@pytest.mark.parametrize("what", [float("inf"), float("nan")])
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D,gap", SIZES)
def test_a_gradient_that_is_not_finite_stays_in_its_row(n, V, D, gap, t, what):
    h, w, target, grad = ops.xent_inputs(n, V, D, t, gap, n)
    x = tt.VocabCrossEntropy(V, D)
    grad = grad.round(decimals=3) * 1000  # beyond what fp16 holds in units of 2^-15
    ref = x.loss_and_grad(h, w, target, grad)
    grad[3] = what
    got = x.loss_and_grad(h, w, target, grad)
    rest = torch.arange(n, device=ops.DEV) != 3
    assert not torch.isfinite(got[2][3]).any()
    assert torch.isfinite(got[2][rest]).all()
    close = (got[2][rest].double() - ref[2][rest].double()).abs() <= 8 * ops.u(t) * ref[2].double().abs().amax()
    assert close.all()


@pytest.mark.parametrize("n,V,D,gap", SIZES)
def test_hidden_rows_of_zeros_beside_tiny_ones(n, V, D, gap):
    h, w, target, grad = ops.xent_inputs(n, V, D, F32, gap, n)
    h = h * 2.0 ** -100
    h[::3] = 0
    z, lse, loss, d, mag = ops.xent_reference(h, w, target, grad, -100)
    got = tt.VocabCrossEntropy(V, D).loss_and_grad(h, w, target, grad)
    ref = d.t() @ h.double()
    h64 = h.double()
    mag = mag + 2.0 ** -17 * grad.double()[:, None]  # d's own floor, as a part of 2^-21
    bound = (2.0 ** -21 + (220 + 6 * (n + 8)) * U32) * (mag.t() @ h64.abs())
    ops.close(got[3], ref, bound + 2.0 ** -38 * n * (grad.double()[:, None] * h64.abs()).max(), "dw")
    assert torch.isfinite(got[2]).all()


def check_entries(n, V, D, gap, seed):
    """Each entry of grad_weight within the roundings that it takes: no bound
    here is near the 2^-11 of a single fp16 term."""
    h, w, target, grad = ops.xent_inputs(n, V, D, F32, gap, seed)
    got = tt.VocabCrossEntropy(V, D).loss_and_grad(h, w, target, grad)
    z, lse, _, d, mag = ops.xent_reference(h, w, target, grad, -100)
    h64, size = h.double(), grad.double()[:, None]
    ez = (6 * D + 8) * U32 * (h64.abs() @ w.double().abs().t()).amax(1)
    es = 2 * ez + U32 * (208 + V / 1024 + 4 * (z - lse[:, None]).abs().amax(1))
    bound = (2.0 ** -21 + es[:, None]) * mag + 2.0 ** -38 * size
    floor = 2.0 ** -38 * n * (size * h64.abs()).amax()
    ref = d.t() @ h64
    ops.close(got[3], ref, bound.t() @ h64.abs() + 6 * (n + 8) * U32 * (mag.t() @ h64.abs()) + U32 * ref.abs() + floor,
              "dw")


@pytest.mark.parametrize("n,V,D,gap", [(9, 796, 17, 0), (7, 10700, 19, 1), (134, 92616, 4, 8), (136, 116602, 36, 1),
                                       (20, 40000, 128, 0), (60, 9000, 256, 0), (200, 3000, 600, 3)])
def test_both_terms_of_every_entry(n, V, D, gap):
    # gradients of the rows that are no powers of two, over many entries
    for seed in range(4):
        check_entries(n, V, D, gap, seed)


@pytest.mark.parametrize("n", [1, 5, 33, 64, 128, 129, 300])
@pytest.mark.parametrize("V,D", [(2000, 40), (2000, 128), (2000, 160), (900, 600)])
def test_probabilities_add_up_where_logits_are_inexact(n, V, D):
    # d is exp(z - lse) - [v = target]: its sum over the vocabulary, which a
    # column of ones in the weight gives, is 0 whatever the rounding of z, as
    # long as lse is that of the same z.  Hidden rows share a large part u that
    # the weight's rows have (almost) nothing of: z is small, its terms are not.
    g = ops.gen(n + D)
    u = torch.randn(D, device=ops.DEV, generator=g, dtype=torch.float64)
    u[D - 1] = 0
    w = torch.randn((V, D), device=ops.DEV, generator=g, dtype=torch.float64) * 2 / D ** 0.5
    w[:, D - 1] = 0
    w -= (w @ u)[:, None] * u / (u @ u)
    target = torch.randint(0, V, (n,), device=ops.DEV, generator=g)
    h = torch.randn((n, D), device=ops.DEV, generator=g, dtype=torch.float64)
    h += 14 * w[target] / w[target].square().sum(1, keepdim=True) + 5000 * u
    h[:, D - 1], w[:, D - 1] = 0, 1
    h, w, grad = h.float(), w.float(), torch.rand(n, device=ops.DEV, generator=g) + 0.5
    z, lse, loss, d, _ = ops.xent_reference(h, w, target, grad, -100)
    got = tt.VocabCrossEntropy(V, D).loss_and_grad(h, w, target, grad)
    p = (z - lse[:, None]).exp()
    size = d.abs().sum(1)
    # the roundings of lse, of the exponentials on both sides, of d and of the sum over V
    one = (208 + V / 1024 + 2 * lse.abs() + 4 * (p * ((z - lse[:, None]).abs() + 1)).sum(1)) * U32
    bound = grad * (one + V * 2.0 ** -38) + (2.0 ** -21 + 6 * (V + 8) * U32) * size
    off = got[2][:, D - 1].double().abs()
    assert (off <= bound).all(), float((off - bound).max())
