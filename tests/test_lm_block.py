"""The norms between two blocks with gate and residual, forward and backward,
against plain 64-bit forms and differences.

Tolerances: a row's sum of D <= 16384 terms takes at most 16 additions in a
thread, 6 across a wave and 16 across waves, so a mean or a mean square is off
by less than 64 x 2^-24 of the terms' magnitudes, and so is what follows from
it by a few roundings; the backward goes through four such sums in a row: 256 x
2^-24.  Sums over n rows add n x 2^-24 of theirs, a type's rounding eps / 2 of
the value (fp16: or half of its smallest step)."""

import pytest
import test_lm_abi as abi
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

F32, BF16, F16, U32, DEV = ops.F32, ops.BF16, ops.F16, ops.U32, ops.DEV
ARG, WS, UNSUPPORTED = abi.ARG, abi.WS, abi.UNSUPPORTED
P, Q, R = abi.P, abi.Q, abi.R
EPS = 1e-5

# ----------------------------------------------------------------- refusals

FWD = dict(x=P, ld_x=8, r=Q, ld_r=8, n=4, D=8, dtype=1, rdt=0, gate=R, ld_gate=0, pg=P, pb=P, g=P, b=P, pdt=0, kind=2,
           eps=1e-5, sr=1.0, sb=1.0, y=R, ld_y=8, h=R, ld_h=8, stats=None, stream=None)
BWD = dict(gy=P, ld_gy=8, gh=None, ld_gh=0, x=P, ld_x=8, r=Q, ld_r=8, n=4, D=8, dtype=1, rdt=0, gate=R, ld_gate=0, pg=P,
           pb=P, g=P, pdt=0, kind=2, sr=1.0, sb=1.0, stats=P, gx=R, ld_gx=8, gr=R, ld_gr=8, gg=None, ld_gg=0, dpg=None,
           dpb=None, dg=None, db=None, ws=abi.W, ws_bytes=300, stream=None)


def test_entry_points_refuse():
    for bad in (dict(x=None), dict(x=P + 1), dict(r=None), dict(r=Q + 2), dict(ld_x=7), dict(ld_r=7), dict(n=-1),
                dict(D=0), dict(dtype=3), dict(rdt=2), dict(pdt=2), dict(kind=8), dict(kind=-1), dict(kind=3),
                dict(kind=0), dict(gate=R + 2), dict(kind=6, gate=None),
                dict(kind=6, ld_gate=7), dict(kind=6, gate=R + 1, ld_gate=8), dict(pg=P + 2), dict(pb=P + 2),
                dict(g=P + 2)):
        assert abi.call("tt_emb_block_forward", FWD, **bad) == ARG, bad
        assert abi.call("tt_emb_block_backward", BWD, **bad) == ARG, bad
    for bad in (dict(y=None), dict(h=None), dict(ld_y=7), dict(ld_h=7), dict(eps=-1.0), dict(eps=float("nan")),
                dict(b=P + 2), dict(kind=1, pg=None, pb=None), dict(stats=P + 2), dict(h=R + 2)):
        assert abi.call("tt_emb_block_forward", FWD, **bad) == ARG, bad
    for bad in (dict(gy=None), dict(ld_gy=7), dict(gh=P, ld_gh=7), dict(gh=P + 2, ld_gh=8), dict(stats=None),
                dict(stats=P + 2), dict(gx=None), dict(gr=None), dict(ld_gx=7), dict(ld_gr=7), dict(gg=P + 2),
                dict(kind=6, ld_gate=8, gg=None), dict(kind=6, ld_gate=8, gg=P, ld_gg=7), dict(dg=P + 2),
                dict(kind=0, pg=None, pb=None, dpg=P)):
        assert abi.call("tt_emb_block_backward", BWD, **bad) == ARG, bad
    for bad in (dict(), dict(ws=None, ws_bytes=1 << 30), dict(ws=abi.W + 8, ws_bytes=1 << 30)):
        assert abi.call("tt_emb_block_backward", BWD, **bad) == WS, bad
    big = dict(D=16385, ld_x=16385, ld_r=16385)
    assert abi.call("tt_emb_block_forward", FWD, ld_y=16385, ld_h=16385, **big) == UNSUPPORTED
    assert abi.call("tt_emb_block_backward", BWD, n=2 ** 31) == UNSUPPORTED


def test_binding_refuses():
    abi.refused(tt.BlockNorm, 8, kind="batch", msg="kind")
    with pytest.raises(tt.TTEmbError):
        tt.BlockNorm(16385)
    x, v = torch.zeros(4, 8), torch.zeros(8)
    b = tt.BlockNorm(8)
    abi.refused(b.forward, x, x, msg="GPU")
    abi.refused(b.forward, torch.zeros(4, 7), x, msg="shape")
    abi.refused(b.forward, x.double(), x, msg="GPU")
    abi.refused(b.backward, x, x, x, x, torch.zeros(4, 4), msg="GPU")
    assert v.numel() == 8


# ------------------------------------------------------------------ results

def make(n, D, t, r, kind, post, gate, p, gap, seed):
    g = ops.gen(seed)
    x, res = ops.rows(g, n, D, t, gap), ops.rows(g, n, D, r, gap, 2.0)
    res += 3.0
    vec = lambda at: (at + 0.2 * torch.randn(D, device=DEV, generator=g)).to(p)  # noqa: E731
    layer = kind == "layer"
    kw = dict(gamma=vec(1.0), beta=vec(0.0) if layer else None, post_gamma=vec(1.0) if post else None,
              post_beta=vec(0.0) if post and layer else None,
              gate=None if gate is None else vec(0.5) if gate == "vector" else ops.rows(g, n, D, t, gap))
    return x, res, kw, ops.rows(g, n, D, t, gap), ops.rows(g, n, D, r, gap)


def norm64(v, layer, D):
    c = v - v.mean(1, keepdim=True) if layer else v
    rstd = (c.square().mean(1, keepdim=True) + EPS).rsqrt()
    return c * rstd, rstd


def forward64(x, res, kw, layer, post, a, b):
    """y, h and what bounds their errors are multiples of."""
    D = x.shape[1]
    k = {q: None if v is None else v.double() for q, v in kw.items()}
    one = lambda v: 1.0 if v is None else v  # noqa: E731
    zero = lambda v: 0.0 if v is None else v  # noqa: E731
    u, mu = x, x.abs()
    if post:
        xhat, rx = norm64(x, layer, D)
        u = xhat * one(k["post_gamma"]) + zero(k["post_beta"])
        mu = one(k["post_gamma"]) * 1.0
        mu = (xhat.abs() + 1 + rx * x.abs().mean(1, keepdim=True)) * (mu.abs() if torch.is_tensor(mu) else mu)
        mu = mu + (k["post_beta"].abs() if k["post_beta"] is not None else 0.0)
    w = b * one(k["gate"])
    h = a * res + w * u
    mh = (a * res).abs() + (w.abs() if torch.is_tensor(w) else abs(w)) * mu
    hhat, rh = norm64(h, layer, D)
    y = hhat * one(k["gamma"]) + zero(k["beta"])
    my = ((hhat.abs() + 1) * (1 + rh * mh.mean(1, keepdim=True)) + rh * mh)
    my = my * (k["gamma"].abs() if k["gamma"] is not None else 1.0)
    return y, h, my + (k["beta"].abs() if k["beta"] is not None else 0.0), mh


CASES = [(1, 1, 0), (3, 2, 0), (5, 7, 3), (17, 128, 0), (33, 129, 1), (4, 512, 0), (70, 513, 0), (9, 1001, 5),
         (700, 1024, 0), (1300, 640, 2), (20, 2048, 0), (6, 2049, 0), (7, 4096, 0), (40, 4100, 4),
         (3, 8192, 0), (5, 8200, 8), (2, 16384, 0),
         (35, 9999, 0), (3000, 24, 0), (1500, 300, 0), (2, 5, 1), (1100, 3000, 0), (2100, 4099, 0)]
KINDS = [(F32, F32, F32), (BF16, BF16, F32), (BF16, F32, BF16), (F16, F16, F16), (F16, F32, F32)]


@pytest.mark.gpu
@pytest.mark.parametrize("t,r,p", KINDS)
@pytest.mark.parametrize("n,D,gap", CASES)
def test_forward_and_gradients(n, D, gap, t, r, p):
    which = CASES.index((n, D, gap)) + KINDS.index((t, r, p))
    for i, (kind, post, gate) in enumerate((("layer", True, "vector"), ("rms", True, "rows"), ("rms", False, None),
                                            ("layer", False, "rows"), ("rms", True, "vector"))):
        if i != which % 5 and i != (which + 2) % 5:
            continue
        print(f"[case] block n={n} D={D} gap={gap} {t} {r} {p} {kind} post={post} gate={gate}", flush=True)
        layer, a, b = kind == "layer", 1.25, 0.7
        x, res, kw, gy, gh = make(n, D, t, r, kind, post, gate, p, gap, n + D)
        op = tt.BlockNorm(D, kind=kind, post=post, eps=EPS, residual_scale=a, block_scale=b)
        y, h, stats = op.forward(x, res, **kw)
        leaves = {"x": x, "residual": res, **{k: v for k, v in kw.items() if v is not None}}
        leaves = {k: v.double().requires_grad_() for k, v in leaves.items()}
        params = {k: leaves.get(k) for k in kw}
        y64, h64, my, mh = forward64(leaves["x"], leaves["residual"], params, layer, post, a, b)
        tiny = lambda k: 2.0 ** -25 if k == F16 else 0.0  # noqa: E731
        ops.close(h, h64.detach(), 64 * U32 * mh.detach() + ops.u(r) * 1.01 * h64.detach().abs() + tiny(r), "h")
        ops.close(y, y64.detach(), 64 * U32 * my.detach() + ops.u(t) * 1.01 * y64.detach().abs() + tiny(t), "y")
        back = {k: v for k, v in kw.items() if k != "beta"}
        for given in (gh, None):
            got = op.backward(gy, given, x, res, stats, **back)
            loss = (gy.double() * y64).sum() + (0.0 if given is None else (given.double() * h64).sum())
            grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()), retain_graph=True)))
            # magnitudes of the gradients' terms
            hhat, rh = norm64(h64.detach(), layer, D)
            xhat, rx = norm64(x.double(), layer, D) if post else (x.double(), 1.0)
            k = {q: None if v is None else v.double().abs() for q, v in kw.items()}
            one = lambda v: 1.0 if v is None else v  # noqa: E731
            amp = 1 + (rh * mh.detach()).amax(1, keepdim=True)  # what an error of h is worth in N(h)
            q = gy.double().abs() * one(k["gamma"])
            mdh = rh * (q + (1 + hhat.abs()) * (1 + hhat.abs().amax(1, keepdim=True)) * q.mean(1, keepdim=True))
            mdh = mdh * amp + (0.0 if given is None else given.double().abs())
            mdu = b * one(k["gate"]) * mdh
            mu = (xhat.abs() + 1 + rx * x.double().abs().mean(1, keepdim=True)) * one(k["post_gamma"]) \
                + (0.0 if k["post_beta"] is None else k["post_beta"]) if post else x.double().abs()
            mdx = mdu
            if post:
                z = mdu * one(k["post_gamma"])
                peak = 1 + xhat.abs().amax(1, keepdim=True) + rx * x.double().abs().mean(1, keepdim=True)
                mdx = rx * (z + (1 + xhat.abs()) * peak * z.mean(1, keepdim=True))
            sums = 256 + n
            bounds = {"x": (256 * U32 * mdx, t), "residual": (256 * U32 * a * mdh, r)}
            if gate == "rows":
                bounds["gate"] = (256 * U32 * b * mdh * mu, t)
            elif gate:
                bounds["gate"] = ((sums * U32 * b * mdh * mu).sum(0), p)
            big = (1 + hhat.abs()) * amp
            bounds["gamma"] = ((sums * U32 * gy.double().abs() * big).sum(0), p)
            if layer:
                bounds["beta"] = ((sums * U32 * gy.double().abs()).sum(0), p)
            if post:
                bounds["post_gamma"] = ((sums * U32 * mdu * mu / one(k["post_gamma"])).sum(0)
                                        + (sums * U32 * mdu * (1 + xhat.abs())).sum(0), p)
                if layer:
                    bounds["post_beta"] = ((sums * U32 * mdu).sum(0), p)
            names = ("x", "residual", "gate", "gamma", "beta", "post_gamma", "post_beta")
            for name, value in zip(names, got):
                assert (value is not None) == (name in bounds), name
                if value is not None:
                    bound, kind_of = bounds[name]
                    assert value.dtype == kind_of
                    ops.close(value, grads[name], bound + ops.u(kind_of) * 1.01 * grads[name].abs() + tiny(kind_of),
                              name)
            again = op.backward(gy, given, x, res, stats, **back)
            assert all(p_ is None or torch.equal(p_, q_) for p_, q_ in zip(got, again))
        assert op.poll_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind,post,gate", [("rms", True, "vector"), ("layer", True, "rows"), ("layer", False, None)])
@pytest.mark.parametrize("D", [40, 4200])
def test_gradients_against_differences(kind, post, gate, D):
    # the derivative along a random direction, by differences of the kernels'
    # own fp32 outputs.  Step 2^-6 of inputs of size 1: the third derivative
    # adds some 2^-12 x 10 of the gradient's size, the outputs' rounding
    # 2^-24 x 2^6 of the loss terms' root of squares: 1e-2 and 1e-5 of them
    n = 6
    x, res, kw, gy, gh = make(n, D, F32, F32, kind, post, gate, F32, 0, 7)
    op = tt.BlockNorm(D, kind=kind, post=post, eps=EPS, block_scale=0.9)
    inputs = {"x": x, "residual": res, **{k: v for k, v in kw.items() if v is not None}}

    def loss(values):
        values = dict(values)
        y, h, stats = op.forward(values.pop("x"), values.pop("residual"), **values)
        return (gy.double() * y.double()).sum() + (gh.double() * h.double()).sum(), stats

    stats = loss(inputs)[1]
    grads = op.backward(gy, gh, x, res, stats, **{k: v for k, v in kw.items() if k != "beta"})
    names = ("x", "residual", "gate", "gamma", "beta", "post_gamma", "post_beta")
    g = ops.gen(11)
    for name, grad in zip(names, grads):
        if grad is None:
            continue
        step = torch.randn(grad.shape, device=DEV, generator=g) * 2.0 ** -6
        up, down = (loss({**inputs, name: inputs[name] + s * step})[0] for s in (1, -1))
        want = float((grad.double() * step.double()).sum())
        scale = float(grad.double().norm() * step.double().norm()) / grad.numel() ** 0.5
        noise = 2 * U32 * 8 * float((gy.double().square().sum() + gh.double().square().sum()).sqrt()) * 4
        assert abs(float(up - down) / 2 - want) <= 1e-2 * (abs(want) + scale) + noise, name


@pytest.mark.gpu
@pytest.mark.parametrize("D", [24, 700, 9000])
def test_rows_do_not_meet(D):
    # rows of NaN and infinity, and rows of zeros, beside ordinary ones
    n = 40
    x, res, kw, gy, gh = make(n, D, F32, F32, "layer", True, "vector", F32, 0, 3)
    op = tt.BlockNorm(D, kind="layer", post=True, eps=EPS)
    y, h, stats = op.forward(x, res, **kw)
    back = {k: v for k, v in kw.items() if k != "beta"}
    ref = op.backward(gy, gh, x, res, stats, **back)
    x2, res2 = x.clone(), res.clone()
    x2[3, 5], res2[7, 0], x2[11], res2[11], x2[20] = float("nan"), float("inf"), 0.0, 0.0, 1e30
    y2, h2, stats2 = op.forward(x2, res2, **kw)
    got = op.backward(gy, gh, x2, res2, stats2, **back)
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[[3, 7, 11, 20]] = False
    assert torch.equal(y2[keep], y[keep]) and torch.equal(h2[keep], h[keep])
    assert torch.equal(got[0][keep], ref[0][keep]) and torch.equal(got[1][keep], ref[1][keep])
    assert bool(y2[3].isnan().all()) and bool(y2[7].isnan().all()) and bool(y2[11].isfinite().all())


@pytest.mark.gpu
def test_no_rows_in_place_and_views():
    D = 72
    op = tt.BlockNorm(D, kind="layer", post=True)
    none = torch.zeros((0, D), device=DEV)
    v = torch.ones(D, device=DEV, dtype=F32)
    y, h, stats = op.forward(none, none, gate=v, gamma=v, beta=v, post_gamma=v, post_beta=v)
    assert y.shape == h.shape == (0, D) and stats.shape == (0, 4)
    got = op.backward(none, none, none, none, stats, gate=v, gamma=v, post_gamma=v, post_beta=v)
    assert got[0].shape == (0, D) and all((q == 0).all() and q.shape == (D,) for q in got[2:])
    # the residual stream updated in place, y over x
    x, res, kw, _, _ = make(300, D, BF16, F32, "layer", True, "vector", F32, 5, 1)
    ref = op.forward(x, res, **kw)
    x2, res2 = (torch.zeros((300, D + 5), device=DEV, dtype=q.dtype)[:, :D].copy_(q) for q in (x, res))
    got = op.forward(x2, res2, out=x2, out_h=res2, **kw)
    assert got[0] is x2 and got[1] is res2 and all(torch.equal(p, q) for p, q in zip(got, ref))
    # without parameters
    y, h, stats = op.forward(x, res)
    want = torch.nn.functional.layer_norm(res.double() + torch.nn.functional.layer_norm(x.double(), (D,)), (D,))
    ops.close(y, want, ops.u(BF16) * 1.01 * want.abs() + 1e-4, "plain")
    dx = op.backward(y, None, x, res, stats)
    assert dx[2] is None and dx[3].dtype == F32


@pytest.mark.gpu
def test_arguments_that_do_not_fit():
    D = 16
    x, v = torch.zeros((4, D), device=DEV, dtype=BF16), torch.ones(D, device=DEV)
    op, layer = tt.BlockNorm(D), tt.BlockNorm(D, kind="layer")
    for kw, msg in ((dict(beta=v), "beta"), (dict(post_gamma=v), "post"), (dict(gamma=v[:8]), "shape"),
                    (dict(gamma=v.half()), "dtype"), (dict(gate=torch.ones((3, D), device=DEV, dtype=BF16)), "shape"),
                    (dict(gate=torch.ones((4, D), device=DEV)), "dtype"), (dict(gate=v.bfloat16(), gamma=v), "dtype"),
                    (dict(out=x[:2]), "shape"), (dict(out_h=x.float()), "dtype"),
                    (dict(gate=x[:, :1].expand(4, D)), "strides")):
        abi.refused(op.forward, x, x, msg=msg, **kw)
    abi.refused(op.forward, x, x.half(), msg="residual")
    abi.refused(layer.forward, x, x, gamma=v, beta=v.bfloat16(), msg="dtype")
    y, h, stats = op.forward(x, x)
    abi.refused(op.backward, x.float(), None, x, x, stats, msg="dtype")
    abi.refused(op.backward, x, x.float(), x, x, stats, msg="dtype")
    abi.refused(op.backward, x, None, x, x, stats[:, :2], msg="shape")
    abi.refused(op.backward, x, None, x, x, torch.zeros((4, 8), device=DEV)[:, :4], msg="contiguous")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 5000])
def test_captured_and_on_another_stream(D):
    n = 200
    x, res, kw, gy, gh = make(n, D, BF16, BF16, "rms", True, "vector", F32, 0, 5)
    op = tt.BlockNorm(D, post=True)

    def step(stream=None):
        y, h, stats = op.forward(x, res, stream=stream, **kw)
        return (y, h) + tuple(q for q in op.backward(gy, gh, x, res, stats, stream=stream, gate=kw["gate"],
                                                     gamma=kw["gamma"], post_gamma=kw["post_gamma"])
                              if q is not None)

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
        x.mul_(1.5)
        gy.add_(0.25)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(step(), got))
