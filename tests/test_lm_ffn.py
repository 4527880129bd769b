"""The gated feed-forward block, forward and backward, against plain 64-bit
forms and differences.

Tolerances, elementwise, with u = eps / 2 of the type and every product's
magnitudes taken from the absolute values of its operands: a sum of k products
in fp32 is off by at most (k + 8) 2^-24 of them (fp32 operands are three bf16
terms: the dropped products are below 2^-24); the activations and their slopes by
32 x 2^-24 of the terms they are made of, and their slopes stay below 1.13; a and
p's gradient are rounded once (u of the value), and so is what is returned (p to fp32)."""

import pytest
import test_lm_abi as abi
import test_lm_ops as ops
import test_lm_threads as threads
import torch

import tensor_train_compressed_gather_amd as tt

F32, BF16, F16, U32, DEV = ops.F32, ops.BF16, ops.F16, ops.U32, ops.DEV
ARG, WS, UNSUPPORTED = abi.ARG, abi.WS, abi.UNSUPPORTED
P, Q, R = abi.P, abi.Q, abi.R
ACTS = ("silu", "gelu", "gelu_tanh")

# ----------------------------------------------------------------- refusals

FWD = dict(x=P, ld_x=8, w_in=Q, ld_in=8, w_out=R, ld_out=16, n=4, D=8, F=16, dtype=1, act=0, pre=None, ld_pre=32, y=P,
           ld_y=8, ws=abi.W, ws_bytes=300, stream=None)
BWD = dict(gy=P, ld_gy=8, x=P, ld_x=8, pre=Q, ld_pre=32, w_in=Q, ld_in=8, w_out=R, ld_out=16, n=4, D=8, F=16, dtype=1,
           act=0, gx=P, ld_gx=8, gin=P, ld_gin=8, gout=P, ld_gout=16, ws=abi.W, ws_bytes=300, stream=None)


def test_entry_points_refuse():
    for name, good in (("tt_emb_ffn_forward", FWD), ("tt_emb_ffn_backward", BWD)):
        for bad in (dict(x=None), dict(x=P + 1), dict(w_in=None), dict(w_out=None), dict(w_in=Q + 1), dict(ld_x=7),
                    dict(ld_in=7), dict(ld_out=15), dict(n=-1), dict(D=0), dict(F=0), dict(dtype=3), dict(act=3),
                    dict(act=-1), dict(pre=Q + 2), dict(pre=Q, ld_pre=31)):
            assert abi.call(name, good, **bad) == ARG, bad
        for bad in (dict(n=2 ** 31), dict(D=65537, ld_x=65537, ld_in=65537), dict(F=65537, ld_out=65537),
                    dict(n=2 ** 30, F=65536, ld_out=65536)):
            assert abi.call(name, good, **bad) == UNSUPPORTED, bad
        for bad in (dict(), dict(ws=None, ws_bytes=1 << 40), dict(ws=abi.W + 16, ws_bytes=1 << 40)):
            assert abi.call(name, good, **bad) == WS, bad
    for bad in (dict(y=None), dict(ld_y=7), dict(y=P + 1)):
        assert abi.call("tt_emb_ffn_forward", FWD, **bad) == ARG, bad
    for bad in (dict(gy=None), dict(ld_gy=7), dict(pre=None), dict(gx=None), dict(gin=None), dict(gout=None),
                dict(ld_gx=7), dict(ld_gin=7), dict(ld_gout=15), dict(gin=P + 1)):
        assert abi.call("tt_emb_ffn_backward", BWD, **bad) == ARG, bad


def size(n, D, F, dtype, what):
    out = abi.C.c_size_t()
    assert tt.lib().tt_emb_ffn_workspace_size(n, D, F, dtype, what, abi.C.byref(out)) == 0
    return out.value


def test_sizes():
    out = abi.C.c_size_t()
    for bad, code in (((4, 8, 16, 1, 4), ARG), ((4, 8, 16, 1, -1), ARG), ((4, 0, 16, 1, 0), ARG),
                      ((4, 8, 16, 5, 0), ARG), ((4, 65537, 16, 1, 0), UNSUPPORTED)):
        assert tt.lib().tt_emb_ffn_workspace_size(*bad, abi.C.byref(out)) == code
    assert tt.lib().tt_emb_ffn_workspace_size(4, 8, 16, 1, 0, None) == ARG
    # operands that serve in place take no room: a, and the parts of the sums
    n, D, F = 512, 1024, 4096
    assert size(n, D, F, 1, 2) < size(n, D, F, 1, 0) - (3 * F * D + n * D) * 2 + 4096
    assert size(n, D, F, 0, 2) == size(n, D, F, 0, 0)
    assert size(n, D + 8, F, 1, 2) == size(n, D + 8, F, 1, 2 | 0) > size(n, D, F, 1, 2) + 2 * F * D * 2
    # a workspace for operands in place is refused where one needs a copy
    good = dict(FWD, n=n, D=D, F=F, ld_x=D, ld_in=D, ld_out=F, ld_y=D, ld_pre=2 * F, ws_bytes=size(n, D, F, 1, 2))
    for bad in (dict(x=P + 2), dict(w_in=Q + 8), dict(w_out=R + 2), dict(ld_x=D + 4), dict(ld_in=D + 1),
                dict(ld_out=(1 << 20) + 8)):
        assert abi.call("tt_emb_ffn_forward", good, **bad) == WS, bad
    good = dict(BWD, n=n, D=D, F=F, ld_gy=D, ld_x=D, ld_in=D, ld_out=F, ld_gx=D, ld_gin=D, ld_gout=F, ld_pre=2 * F,
                ws_bytes=size(n, D, F, 1, 3))
    for bad in (dict(gy=P + 2), dict(x=P + 2), dict(w_in=Q + 8), dict(w_out=R + 2), dict(ld_gy=D + 4)):
        assert abi.call("tt_emb_ffn_backward", good, **bad) == WS, bad


def test_binding_refuses():
    abi.refused(tt.GatedFeedForward, 8, 16, activation="relu", msg="activation")
    for bad in ((0, 8), (8, 0)):
        abi.refused(tt.GatedFeedForward, *bad, msg="")
    with pytest.raises(tt.TTEmbError):
        tt.GatedFeedForward(8, 65537)
    op, x = tt.GatedFeedForward(8, 16), torch.zeros(4, 8)
    abi.refused(op.forward, x, torch.zeros(32, 8), torch.zeros(8, 16), msg="GPU")
    abi.refused(op.forward, torch.zeros(4, 9), torch.zeros(32, 8), torch.zeros(8, 16), msg="shape")


# ------------------------------------------------------------------ results

def act64(kind, z):
    if kind == "silu":
        return torch.nn.functional.silu(z)
    if kind == "gelu":  # (1 + erf would lose values below 2^-53)
        return 0.5 * z * torch.erfc(-z * 0.5 ** 0.5)
    return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))


def make(n, D, F, t, gap, seed, std=1.0):
    g = ops.gen(seed)
    x, gy = ops.rows(g, n, D, t, gap), ops.rows(g, n, D, t, gap, 0.3)
    return (x, ops.rows(g, 2 * F, D, t, gap, std / D ** 0.5), ops.rows(g, D, F, t, gap, 1.0 / F ** 0.5), gy)


def check(n, D, F, t, gap, kind, seed=None, terms=1):
    x, w_in, w_out, gy = make(n, D, F, t, gap, n + D + F if seed is None else seed, 2.0)
    op = tt.GatedFeedForward(D, F, activation=kind)
    y, pre = op.forward(x, w_in, w_out, keep=True)
    assert torch.equal(op.forward(x, w_in, w_out), y)
    u, tiny = max(ops.u(t), U32) * 1.01, 2.0 ** -25 if t == F16 else 0.0
    ua = u ** terms  # a and dp: what a term leaves is rounded once more
    X, WI, WO, GY = (v.double() for v in (x, w_in, w_out, gy))
    p = X @ WI.t()
    size_p = X.abs() @ WI.abs().t()
    dp = (D + 8) * U32 * size_p
    assert pre.dtype == F32
    ops.close(pre, p, dp, "p")
    a64 = act64(kind, p[:, :F])
    a = a64 * p[:, F:]
    da = 1.13 * dp[:, :F] * p[:, F:].abs() + (a64.abs() + dp[:, :F]) * dp[:, F:] \
        + 32 * U32 * (p[:, :F] * p[:, F:]).abs() + ua * a.abs() + tiny
    ops.close(y, a @ WO.t(), da @ WO.abs().t() + (F + 8) * U32 * (a.abs() @ WO.abs().t())
              + u * (a @ WO.t()).abs() + tiny, "y")
    del p, size_p, dp, a64, a, da
    # the gradients at the p that the forward gave
    got = op.backward(gy, x, pre, w_in, w_out)
    z = pre.double()[:, :F].requires_grad_()
    up = pre.double()[:, F:]
    v = act64(kind, z)
    slope, = torch.autograd.grad(v.sum(), z)
    z, v = z.detach(), v.detach()
    G = GY @ WO
    eG = (D + 8) * U32 * (GY.abs() @ WO.abs())
    g, h = G * up * slope, G * v
    eg = eG * (up * slope).abs() + 32 * U32 * (G * up).abs() * (1 + z.abs()) + ua * g.abs() + tiny
    eh = eG * v.abs() + 32 * U32 * (G * z).abs() + ua * h.abs() + tiny
    dP, eP = torch.cat([g, h], 1), torch.cat([eg, eh], 1)
    mid, emid = v * up, (ua + 32 * U32) * (v * up).abs() + 32 * U32 * (z * up).abs() + tiny
    for name, value, ref, bound in (
            ("grad_x", got[0], dP @ WI, eP @ WI.abs() + (2 * F + 8) * U32 * (dP.abs() @ WI.abs())),
            ("grad_w_in", got[1], dP.t() @ X, eP.t() @ X.abs() + (n + 8) * U32 * (dP.abs().t() @ X.abs())),
            ("grad_w_out", got[2], GY.t() @ mid,
             GY.abs().t() @ emid + (n + 8) * U32 * (GY.abs().t() @ mid.abs()))):
        assert value.dtype == t
        ops.close(value, ref, bound + u * ref.abs() + tiny, name)
    again = op.backward(gy, x, pre, w_in, w_out)
    assert all(torch.equal(q, r) for q, r in zip(got, again))
    assert op.poll_error() == 0


SHAPES = [(1, 1, 1, 0), (1, 64, 64, 0), (2, 8, 40, 0), (3, 17, 5, 3), (5, 100, 33, 1), (31, 128, 64, 0),
          (64, 64, 128, 8), (12, 1000, 4096, 0), (65, 130, 250, 0), (127, 256, 129, 0),
          (128, 72, 96, 0), (129, 264, 320, 8),
          (200, 1000, 70, 0), (257, 520, 300, 5), (600, 96, 1100, 0), (40, 2000, 3000, 0), (1030, 200, 200, 1),
          (16, 640, 1280, 0), (17, 192, 2048, 0), (9, 4096, 100, 0), (33, 200, 5000, 0),
          (100, 1024, 1500, 0), (4, 130, 9000, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F32, BF16, F16])
@pytest.mark.parametrize("n,D,F,gap", SHAPES)
def test_forward_and_gradients(n, D, F, gap, t):
    kind = ACTS[(SHAPES.index((n, D, F, gap)) + [F32, BF16, F16].index(t)) % 3]
    print(f"[case] ffn n={n} D={D} F={F} gap={gap} {t} {kind}", flush=True)
    check(n, D, F, t, gap, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("n,D,F", [(2048, 64, 4096), (4096, 2048, 4160), (4000, 4096, 4096), (8300, 320, 200)])
def test_large_tiles(n, D, F, t):
    if t == F32:
        n, D, F = n // 2, D // 2, F // 2
    print(f"[case] ffn n={n} D={D} F={F} {t}", flush=True)
    check(n, D, F, t, 0, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("n,D,F,gap", [(1, 1, 1, 0), (14, 53, 19, 0), (3, 17, 5, 3), (64, 64, 32, 8), (17, 130, 120, 1),
                                       (16, 640, 128, 0), (1, 4096, 8192, 0), (1, 2000, 1000, 8), (300, 1000, 6, 0),
                                       (2048, 64, 1, 0), (30, 1024, 68, 8), (4, 300, 512, 0)])
def test_few_values_of_a_have_two_terms(n, D, F, gap, t):
    print(f"[case] ffn two terms n={n} D={D} F={F} gap={gap} {t}", flush=True)
    # up to 2^11 values of a, no gradient of more than 2^22 (1 x 4096 x 8192: a has 2^13, w_in's
    # gradient 4096 x 2 x 8192 = 2^26, so one term, whose half step is `u` and not its square)
    check(n, D, F, t, gap, ACTS[n % 3], terms=2 if n * F <= 1 << 11 and D * max(n, 2 * F) <= 1 << 22 else 1)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 40])
def test_long_fp32_sums_are_rounded_once_a_step(n):
    # da sums D = 4000 products, 16 a step: 250 roundings of half a step, 2^-24 at most, of partial sums whose
    # mean square grows evenly: sqrt(250 / 3 / 2) 2^-24 = 3.8e-7 of da.  Four roundings of dp: 2.4e-7; the sum of
    # 120 values, the terms left out (2^-25) and the result's rounding: 2^-23 = 1.2e-7.  Six roundings a step
    # would be 9.5e-7 for da alone
    D, F = 4000, 60
    x, w_in, w_out, gy = make(n, D, F, F32, 0, 4)
    op = tt.GatedFeedForward(D, F)
    _, pre = op.forward(x, w_in, w_out, keep=True)
    dx, dw_in, _ = op.backward(gy, x, pre, w_in, w_out)
    z = pre.double()[:, :F].requires_grad_()
    v = act64("silu", z)
    slope, = torch.autograd.grad(v.sum(), z)
    G = gy.double() @ w_out.double()
    dP = torch.cat([G * pre.double()[:, F:] * slope, G * v.detach()], 1)
    for got, ref in ((dx, dP @ w_in.double()), (dw_in, dP.t() @ x.double())):
        assert (got.double() - ref).norm() <= 8e-7 * ref.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 20])
def test_an_infinite_a_stays_infinite(n):
    # silu(400) 400 is past fp16; the second term of an infinite a is nothing, not a NaN
    D, F = 8, 16
    x = torch.ones((n, D), device=DEV, dtype=F16)
    w_in, w_out = torch.full((2 * F, D), 50.0, device=DEV, dtype=F16), torch.ones((D, F), device=DEV, dtype=F16)
    op = tt.GatedFeedForward(D, F)
    y, pre = op.forward(x, w_in, w_out, keep=True)
    assert (pre == 400).all() and (y == float("inf")).all()
    dx, dw_in, dw_out = op.backward(x, x, pre, w_in, w_out)
    assert (dw_out == float("inf")).all()
    # dp: 8 x 400 of both projections, as silu(400) is 400 and its slope 1
    assert (dw_in == n * 3200.0).all()


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("n,D,F", [(0, 1, 1), (1, 65536, 65536), (2 ** 28, 100, 100), (129, 64, 65536),
                                   (2 ** 20, 128, 512), (17, 1, 1), (10 ** 6, 4096, 1)])
def test_workspace_of_any_size(n, D, F, dtype):
    for what in (0, 1):
        assert 256 <= size(n, D, F, dtype, what | 2) <= size(n, D, F, dtype, what)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [9, 200])
@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 30])
def test_fp32_keeps_its_precision_at_any_size(n, scale):
    # x times a power of two and the weight by it: the same p; the same for y and
    # the gradient.  All products are those of scale 1, bit for bit
    D, F = 100, 72
    x, w_in, w_out, gy = make(n, D, F, F32, 0, 8)
    op = tt.GatedFeedForward(D, F)
    y, pre = op.forward(x, w_in, w_out, keep=True)
    dx, dw_in, dw_out = op.backward(gy, x, pre, w_in, w_out)
    y2, pre2 = op.forward(x * scale, w_in / scale, w_out * scale, keep=True)
    assert torch.equal(pre, pre2) and torch.equal(y * scale, y2)
    got = op.backward(gy / scale, x * scale, pre2, w_in / scale, w_out * scale)
    assert torch.equal(got[0], dx / scale) and torch.equal(got[1], dw_in * scale)
    assert torch.equal(got[2], dw_out / scale)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ACTS)
def test_activations_over_their_range(kind):
    # D = 1, F = 1: p is x times the two weights; fp32
    z = torch.cat([torch.linspace(-30, 30, 4001), torch.logspace(-30, 2, 200), -torch.logspace(-30, 2, 200)])
    x = z.to(DEV)[:, None].contiguous()
    one = torch.ones((1, 1), device=DEV)
    op = tt.GatedFeedForward(1, 1, activation=kind)
    w_in = torch.tensor([[1.0], [0.0]], device=DEV)
    y, pre = op.forward(x, w_in, one, keep=True)
    assert torch.equal(pre[:, :1], x) and (pre[:, 1] == 0).all() and (y == 0).all()
    pre[:, 1] = 1.0
    leaf = x.double().requires_grad_()
    value = act64(kind, leaf)
    slope, = torch.autograd.grad(value.sum(), leaf)
    dx, _, _ = op.backward(torch.ones_like(x), x, pre, torch.tensor([[1.0], [0.0]], device=DEV), one)
    ops.close(dx, slope, 64 * U32 * (1 + leaf.detach().abs().clamp(max=6)) + 1e-37, "slope")
    dx, _, _ = op.backward(torch.ones_like(x), x, pre, torch.tensor([[0.0], [1.0]], device=DEV), one)
    ref = value.detach()
    ops.close(dx, ref, 32 * U32 * (ref.abs() + (leaf.detach() * slope).abs()) * (1 + leaf.detach().abs()) + 1e-37,
              "value")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("n,D,F", [(7, 40, 24), (150, 129, 200)])
def test_gradients_against_differences(n, D, F, kind):
    # along a random direction: steps of 2^-7 of inputs of size 1 leave a third
    # derivative's 2^-14 x 10 of the change, the outputs' rounding 2^-24 x F of
    # their size over the step
    x, w_in, w_out, gy = make(n, D, F, F32, 0, 5)
    op = tt.GatedFeedForward(D, F, activation=kind)
    pre = op.forward(x, w_in, w_out, keep=True)[1]
    grads = op.backward(gy, x, pre, w_in, w_out)
    g = ops.gen(6)
    for k, grad in enumerate(grads):
        step = torch.randn(grad.shape, device=DEV, generator=g) * 2.0 ** -7 * (1.0, D ** -0.5, F ** -0.5)[k]
        values = []
        for s in (1, -1):
            args = [x, w_in, w_out]
            args[k] = args[k] + s * step
            values.append((gy.double() * op.forward(*args).double()).sum())
        want = float((grad.double() * step.double()).sum())
        size = float(grad.double().norm() * step.double().norm()) / grad.numel() ** 0.5
        noise = 8 * U32 * float(gy.double().norm()) * 4
        assert abs(float(values[0] - values[1]) / 2 - want) <= 5e-3 * (abs(want) + size) + noise, k


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n", [8, 20, 300])
def test_rows_do_not_meet(n, t):
    D, F = 72, 100
    x, w_in, w_out, gy = make(n, D, F, t, 0, 1)
    op = tt.GatedFeedForward(D, F)
    y, pre = op.forward(x, w_in, w_out, keep=True)
    dx = op.backward(gy, x, pre, w_in, w_out)[0]
    x2 = x.clone()
    x2[3, 5], x2[n - 1, 0] = float("nan"), float("inf")
    y2, pre2 = op.forward(x2, w_in, w_out, keep=True)
    dx2 = op.backward(gy, x2, pre2, w_in, w_out)[0]
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[[3, n - 1]] = False
    for a, b in ((y, y2), (pre, pre2), (dx, dx2)):
        assert torch.equal(a[keep], b[keep])
    assert not bool(y2[3].isfinite().any()) and not bool(y2[n - 1].isfinite().any())


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F32, BF16])
def test_no_rows_given_outputs_and_views(t):
    D, F, n = 80, 48, 150
    x, w_in, w_out, gy = make(n, D, F, t, 0, 2)
    op = tt.GatedFeedForward(D, F)
    none = x[:0]
    y, pre = op.forward(none, w_in, w_out, keep=True)
    assert y.shape == (0, D) and pre.shape == (0, 2 * F)
    got = op.backward(none, none, pre, w_in, w_out)
    assert got[0].shape == (0, D) and (got[1] == 0).all() and (got[2] == 0).all()
    y, pre = op.forward(x, w_in, w_out, keep=True)
    ref = op.backward(gy, x, pre, w_in, w_out)

    def inside(a, gap, at):
        flat = torch.full((a.shape[0] * (a.shape[1] + gap) + at + 8,), 7.0, device=DEV, dtype=a.dtype)
        v = flat[at:at + a.shape[0] * (a.shape[1] + gap)].view(a.shape[0], -1)
        v[:, :a.shape[1]] = a
        return flat, v[:, :a.shape[1]]

    for gap, at in ((0, 8), (8, 0), (3, 0), (0, 1), (5, 3)):
        ins = [inside(a, gap, at)[1] for a in (x, w_in, w_out, gy, pre)]
        f1, out = inside(torch.zeros_like(y), gap, at)
        f2, gin = inside(torch.zeros_like(w_in), gap, at)
        f3, gout = inside(torch.zeros_like(w_out), gap, at)
        y2, pre2 = op.forward(*ins[:3], keep=True, out=out)
        assert y2 is out and torch.equal(y2, y) and torch.equal(pre2, pre)
        got = op.backward(ins[3], ins[0], ins[4], ins[1], ins[2], grad_w_in=gin, grad_w_out=gout)
        assert got[1] is gin and got[2] is gout and all(torch.equal(p, q) for p, q in zip(got, ref))
        for flat, v in ((f1, out), (f2, gin), (f3, gout)):  # nothing around them is written
            v.fill_(7.0)
            assert (flat == 7.0).all()


@pytest.mark.gpu
def test_arguments_that_do_not_fit():
    n, D, F = 6, 16, 24
    x, w_in, w_out, gy = make(n, D, F, BF16, 0, 3)
    op = tt.GatedFeedForward(D, F)
    y, pre = op.forward(x, w_in, w_out, keep=True)
    for args, msg in (((x, w_in[:F], w_out), "shape"), ((x, w_in, w_out.t()), "shape"),
                      ((x, w_in.half(), w_out), "dtype"), ((x, w_in, w_out.float()), "dtype"),
                      ((x.double(), w_in, w_out), "dtype"), ((x[0], w_in, w_out), "shape")):
        abi.refused(op.forward, *args, msg=msg)
    abi.refused(op.forward, x, w_in, w_out, out=y[:2], msg="shape")
    abi.refused(op.backward, gy[:2], x, pre, w_in, w_out, msg="shape")
    abi.refused(op.backward, gy, x, pre[:, :F], w_in, w_out, msg="shape")
    abi.refused(op.backward, gy, x, pre.bfloat16(), w_in, w_out, msg="dtype")
    abi.refused(op.backward, gy, x, pre, w_in, w_out, grad_w_in=w_out, msg="shape")


@pytest.mark.gpu
def test_threads_share_an_operator():
    D, F = 64, 200
    op, clip = tt.GatedFeedForward(D, F), tt.GradientClip(0.5)
    cases = [make(n, D, F, BF16, 0, n) for n in (3, 140, 700)]
    refs = []

    def step(x, w_in, w_out, gy):
        y, pre = op.forward(x, w_in, w_out, keep=True)
        grads = list(op.backward(gy, x, pre, w_in, w_out))
        norm = clip.clip(grads)
        return [y, pre, norm, *grads]

    for c in cases:
        refs.append(step(*c))
    torch.cuda.synchronize()

    def work(k):
        for _ in range(15):
            got = step(*cases[k])
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, refs[k]))

    threads.in_threads(work, 3)
    assert op.poll_error() == 0 and clip.poll_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("t,n,D,F", [(BF16, 5, 128, 256), (BF16, 300, 100, 90), (F32, 40, 64, 96)])
def test_captured_and_on_another_stream(t, n, D, F):
    x, w_in, w_out, gy = make(n, D, F, t, 0, 4)
    op = tt.GatedFeedForward(D, F)

    def step(stream=None):
        y, pre = op.forward(x, w_in, w_out, keep=True, stream=stream)
        return (y, pre) + op.backward(gy, x, pre, w_in, w_out, stream=stream)

    ref = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = step(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for k in range(3):
        x.mul_(0.75)
        gy.add_(0.125)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(step(), got))
