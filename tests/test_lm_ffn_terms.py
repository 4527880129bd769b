"""The gated feed-forward block in 16 bits: where a and p's gradient have two
terms, what is returned is off by its own rounding and little else.

With e the returned values' own rounding (of the 64-bit values) and d what the
operator is off by before it, the error is at most |e| + 2 |d| elementwise (the
distance to the nearest value of the type is 1-Lipschitz), so the same holds for
the norms.  d: two terms leave u^2 of a value of a or dp, u = eps / 2, at
random, so u^2 / sqrt(3) of a sum of independent products; the hardware's
exponential and reciprocal some 2^-22; sums of up to 16384 fp32 products at 32 a
step 512 roundings of 2^-24 / sqrt(3).  Together below 1.2e-5 of the sum in
bf16 (2^-16 / sqrt(3) = 0.9e-5) and 1e-6 in fp16.  e is u / sqrt(3) of values spread
evenly between the powers of two, 0.7 u on average over them: 1.6e-3 in bf16, 2e-4 in
fp16.  2 |d| / |e| is 2 % then; four times that for draws of few values: 1.08.
One term: 1.41 as a rule."""

import pytest
import test_lm_ffn as ffn
import torch

import tensor_train_compressed_gather_amd as tt

MOST = 1.08


def ratio(got, ref):
    e = (ref.to(got.dtype).double() - ref).norm()
    return float((got.double() - ref).norm() / e)


def forward64(kind, x, w_in, w_out):
    F = w_out.shape[1]
    p = x.double() @ w_in.double().t()
    return (ffn.act64(kind, p[:, :F]) * p[:, F:]) @ w_out.double().t()


# the longest sums of the fewest outputs, more outputs of few values of a; 17 rows and more go by tiles
FORWARD = [(1, 16, 4096), (2, 24, 2000), (1, 16, 16384), (4, 64, 1000), (1, 300, 6000), (16, 120, 3000),
           (4, 4096, 512), (3, 9000, 64), (1, 9000, 2000), (12, 9000, 170), (17, 16, 3001), (40, 50, 700)]


@pytest.mark.gpu
@pytest.mark.parametrize("t", [ffn.BF16, ffn.F16])
@pytest.mark.parametrize("n,D,F", FORWARD)
def test_few_outputs_are_rounded_once(n, D, F, t):
    kind = ffn.ACTS[F % 3]
    print(f"[case] ffn terms n={n} D={D} F={F} {t} {kind}", flush=True)
    op = tt.GatedFeedForward(D, F, activation=kind)
    for seed in range(12 if n * D < 1000 else 3):
        x, w_in, w_out, _ = ffn.make(n, D, F, t, 0, 100 + seed, 2.0)
        assert ratio(op.forward(x, w_in, w_out), forward64(kind, x, w_in, w_out)) <= MOST, seed


# which of the three gradients has few outputs (or dp and a few values)
BACKWARD = [(1, 16, 4096, "x"), (2, 24, 2000, "x"), (4, 300, 2000, "x"), (17, 16, 3001, "x"), (2000, 8, 16, "io"),
            (30000, 4, 30, "io"), (777, 40, 40, "o"), (100, 3, 300, "xio"), (9, 3000, 200, "xio")]


@pytest.mark.gpu
@pytest.mark.parametrize("t", [ffn.BF16, ffn.F16])
@pytest.mark.parametrize("n,D,F,which", BACKWARD)
def test_gradients_of_few_values_are_rounded_once(n, D, F, which, t):
    kind = ffn.ACTS[F % 3]
    print(f"[case] ffn terms n={n} D={D} F={F} {t} {kind}", flush=True)
    op = tt.GatedFeedForward(D, F, activation=kind)
    for seed in range(4):
        x, w_in, w_out, gy = ffn.make(n, D, F, t, 0, 200 + seed, 2.0)
        _, pre = op.forward(x, w_in, w_out, keep=True)
        got = op.backward(gy, x, pre, w_in, w_out)
        z = pre.double()[:, :F].requires_grad_()
        up = pre.double()[:, F:]
        v = ffn.act64(kind, z)
        slope, = torch.autograd.grad(v.sum(), z)
        v = v.detach()
        G = gy.double() @ w_out.double()
        dP = torch.cat([G * up * slope, G * v], 1)
        refs = {"x": dP @ w_in.double(), "i": dP.t() @ x.double(), "o": gy.double().t() @ (v * up)}
        for name, value in zip("xio", got):
            if name in which:
                assert ratio(value, refs[name]) <= MOST, (name, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [ffn.BF16, ffn.F16])
@pytest.mark.parametrize("n,D,F", [(17, 120, 61000), (65536, 3, 16), (4000, 4096, 1), (16, 128, 65536), (70000, 2, 10),
                                   (1, 65536, 8)])
def test_two_terms_at_the_ends_of_their_range(n, D, F, t):
    # the longest and the widest grids around the rule's bounds, elementwise (one term's bounds hold for two)
    print(f"[case] ffn terms n={n} D={D} F={F} {t}", flush=True)
    ffn.check(n, D, F, t, 0, ffn.ACTS[n % 3])
