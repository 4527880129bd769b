"""The operators around the table (lookup, layer norm, vocabulary cross
entropy, AdamW) against plain 64-bit forms, at the sizes, strides and masks
where they can go wrong.

Tolerances are error bounds, elementwise: a rounding to a type is off by at
most u = eps / 2 of the value, a sum of k terms in fp32 by at most k * 2^-24
of the sum of the terms' magnitudes."""

import math

import pytest
import torch

import tensor_train_compressed_gather_amd as tt

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
U32 = 2.0 ** -24


def u(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows(g, n, D, t, gap=0, std=1.0):
    """[n, D] values in rows that are D + gap elements apart."""
    return (std * torch.randn((n, D + gap), device=DEV, generator=g)).to(t)[:, :D]


def close(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: off by {float(over.max()):.3e} more than the bound"


# ------------------------------------------------------------------- lookup

LOOKUP = [(1, 1, 1, 0), (1, 7, 5, 3), (3, 50, 8, 0), (17, 9, 33, 1), (64, 3, 64, 0), (300, 40, 100, 5),
          (1000, 1, 16, 0), (5000, 1000, 130, 0), (4097, 20, 264, 2), (20000, 300, 72, 8), (700, 5000, 1025, 0)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,V,D,gap", LOOKUP)
def test_lookup_and_gradient(n, V, D, gap, t):
    print(f"[case] lookup n={n} V={V} D={D} gap={gap} {t}", flush=True)
    g = gen(n + V)
    w = rows(g, V, D, t, gap)
    # a few frequent tokens and many rare ones
    tok = (torch.rand(n, device=DEV, generator=g) ** 4 * V).long().clamp_(max=V - 1)
    scale = 1.7
    for pad, add in ((-1, False), (0, True), (int(tok[0]), False)):
        e = tt.TokenEmbedding(V, D, scale=scale, padding_idx=pad)
        out = e.forward(w, tok)
        ref = w.double()[tok] * scale
        s32 = float(torch.tensor(scale, dtype=F32))
        close(out, ref, ref.abs() * (u(t) + 2 * U32 + abs(s32 / scale - 1)) + 2.0 ** -24 * (t == F16), "forward")
        dy = rows(g, n, D, t, gap)
        old = rows(g, V, D, t, gap)
        dw = e.backward(dy, tok, grad_weight=old.clone() if add else None, accumulate=add)
        keep = (tok != pad)[:, None]
        d64 = dy.double() * keep
        total = torch.zeros((V, D), dtype=torch.float64, device=DEV).index_add_(0, tok, d64)
        mag = torch.zeros_like(total).index_add_(0, tok, d64.abs())
        k = torch.bincount(tok, minlength=V).double()[:, None]
        ref = total * scale + (old.double() if add else 0.0)
        bound = (k + 3) * U32 * mag * scale + (u(t) + 2 * U32) * (ref.abs() + 0.01 * mag) + 2.0 ** -24 * (t == F16)
        close(dw, ref, bound, "gradient")
        if not add:
            assert (dw[(k[:, 0] == 0) | (torch.arange(V, device=DEV) == pad)] == 0).all()
        again = e.backward(dy, tok, grad_weight=old.clone() if add else None, accumulate=add)
        assert torch.equal(dw, again)
        assert e.poll_error() == 0


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 63, 64, 65, 96, 97, 128, 200])
def test_lookup_gradient_of_runs_at_tile_edges(n):
    # runs of one token around the 32-position tiles: `head` positions of
    # token 1, `run` of token 5, the rest of token 9; whole numbers sum exactly
    V, D = 12, 40
    e = tt.TokenEmbedding(V, D)
    for head in (0, 1, 5, 31, 32, 33, 64):
        for run in (0, 1, 31, 32, 33, 63, 64, 65, 100):
            if head + run > n:
                continue
            tok = torch.tensor([1] * head + [5] * run + [9] * (n - head - run), device=DEV, dtype=torch.int64)
            tok = tok[torch.randperm(n, device=DEV, generator=gen(n + head + run))]
            dy = torch.randint(-8, 8, (n, D), device=DEV, generator=gen(run)).float()
            ref = torch.zeros((V, D), device=DEV).index_add_(0, tok, dy)
            dw = e.backward(dy, tok)
            assert torch.equal(dw, ref), (n, head, run)


@pytest.mark.parametrize("n,V", [(7, 2 ** 21 + 3), (2048, 2 ** 20), (2049, 2 ** 20 - 1), (2049, 2 ** 20), (4100, 700),
                                 (70000, 5000), (131072, 1023), (131073, 1023), (150000, 2 ** 20 + 77)])
def test_lookup_gradient_of_every_sort(n, V):
    # token counts and vocabularies on both sides of each sort's limits; half
    # of the tokens are few, whole numbers sum exactly
    D = 8
    g = gen(n)
    tok = torch.randint(0, V, (n,), device=DEV, generator=g)
    few = torch.rand(n, device=DEV, generator=g) < 0.5
    tok[few] = tok[few] % 13
    dy = torch.randint(-8, 8, (n, D), device=DEV, generator=g).float()
    e = tt.TokenEmbedding(V, D, padding_idx=3)
    keep = tok != 3
    ref = torch.zeros((V, D), device=DEV).index_add_(0, tok[keep], dy[keep])
    assert torch.equal(e.backward(dy, tok), ref)
    old = torch.randint(-8, 8, (V, D), device=DEV, generator=g).float()
    assert torch.equal(e.backward(dy, tok, grad_weight=old.clone(), accumulate=True), ref + old)


@pytest.mark.parametrize("n,D", [(100, 64), (3000, 130), (9000, 1030), (40000, 36)])
def test_lookup_gradient_of_one_token(n, D):
    dy = torch.randint(-8, 8, (n, D), device=DEV, generator=gen(n)).float()
    dw = tt.TokenEmbedding(5, D).backward(dy, torch.full((n,), 2, device=DEV))
    assert torch.equal(dw[2], dy.sum(0)) and int((dw != 0).any(1).sum()) <= 1


@pytest.mark.parametrize("n", [1, 7, 8, 9, 15, 16, 17, 24, 25, 40])
def test_lookup_gradient_of_short_runs(n):
    # runs of every length up to three tiles of eight, from every place in a tile
    V, D = 12, 16
    e = tt.TokenEmbedding(V, D)
    for head in range(9):
        for run in range(0, n - head + 1):
            tok = torch.tensor([1] * head + [5] * run + [9] * (n - head - run), device=DEV, dtype=torch.int64)
            dy = torch.randint(-8, 8, (n, D), device=DEV, generator=gen(run)).float()
            ref = torch.zeros((V, D), device=DEV).index_add_(0, tok, dy)
            assert torch.equal(e.backward(dy, tok), ref), (n, head, run)


def test_lookup_of_no_tokens():
    e = tt.TokenEmbedding(6, 10)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    assert e.forward(torch.ones((6, 10), device=DEV), none).shape == (0, 10)
    dw = e.backward(torch.zeros((0, 10), device=DEV), none, grad_weight=torch.ones((6, 10), device=DEV))
    assert (dw == 0).all()
    dw = e.backward(torch.zeros((0, 10), device=DEV), none, grad_weight=torch.ones((6, 10), device=DEV),
                    accumulate=True)
    assert (dw == 1).all()


def test_lookup_takes_tokens_of_any_shape():
    e = tt.TokenEmbedding(11, 24, scale=2.0)
    w = rows(gen(1), 11, 24, BF16)
    tok = torch.randint(0, 11, (3, 5), device=DEV)
    out = e.forward(w, tok)
    assert out.shape == (3, 5, 24) and torch.equal(out.view(15, 24), e.forward(w, tok.view(-1)))
    assert torch.equal(e.backward(out, tok), e.backward(out.view(15, 24), tok.view(-1)))


@pytest.mark.parametrize("bad", [-1, 50, 2 ** 40, -2 ** 62])
def test_lookup_reports_tokens_out_of_range(bad):
    V, D, n = 50, 20, 70
    g = gen(3)
    w, dy = rows(g, V, D, F32), rows(g, n, D, F32)
    tok = torch.randint(0, V, (n,), device=DEV, generator=g)
    tok[13] = bad
    e = tt.TokenEmbedding(V, D)
    out = e.forward(w, tok)
    assert (out[13] == 0).all() and torch.equal(out[:13], w[tok[:13]])
    assert e.poll_error() == tt.TT_EMB_ERR_INDEX and e.poll_error() == 0
    dw = e.backward(dy, tok)
    assert e.poll_error() == tt.TT_EMB_ERR_INDEX and e.poll_error() == 0
    keep = torch.arange(n, device=DEV) != 13
    assert torch.equal(dw, e.backward(dy[keep], tok[keep]))
    assert e.poll_error() == 0


def test_lookup_passes_nan_and_infinity_to_their_rows_only():
    e = tt.TokenEmbedding(4, 16)
    w = torch.ones((4, 16), device=DEV)
    w[2, 3], w[3, 0] = float("nan"), float("inf")
    tok = torch.tensor([0, 2, 3, 1, 2], device=DEV)
    out = e.forward(w, tok)
    assert torch.equal(out.isnan(), w[tok].isnan()) and out[2, 0] == float("inf")
    dw = e.backward(out, tok)
    assert torch.equal(dw.isnan(), w.isnan()) and dw[3, 0] == float("inf") and (dw[1] == 1).all()


# --------------------------------------------------------------------- norm

NORM = [(1, 1, 0), (1, 3, 2), (2, 16, 0), (5, 64, 0), (300, 128, 0), (33, 100, 7), (70, 513, 3), (9, 1000, 0),
        (40, 1024, 32), (3000, 264, 0), (7, 2049, 1), (5, 4096, 0), (3, 8192, 0), (2, 10007, 1), (3, 16384, 0)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,D,gap", NORM)
def test_norm_and_gradients(n, D, gap, t):
    print(f"[case] norm n={n} D={D} gap={gap} {t}", flush=True)
    g = gen(n + D)
    x = rows(g, n, D, t, gap, 2.0)
    x += torch.randn((n, 1), device=DEV, generator=g).to(t)
    gamma = (1 + 0.3 * torch.randn(D, device=DEV, generator=g))
    beta = torch.randn(D, device=DEV, generator=g)
    dy = rows(g, n, D, t, gap)
    eps = 1e-3
    op = tt.LayerNorm(D, eps=eps)
    for gm, bt in ((gamma, beta), (gamma.to(t), None), (None, None)):
        y, mean, rstd = op.forward(x, gm, bt)
        x64 = x.double()
        gm64 = torch.ones(D, device=DEV, dtype=torch.float64) if gm is None else gm.double()
        bt64 = torch.zeros(D, device=DEV, dtype=torch.float64) if bt is None else bt.double()
        m64 = x64.mean(1)
        r64 = 1 / (x64.var(1, correction=0) + eps).sqrt()
        xh = (x64 - m64[:, None]) * r64[:, None]
        big = x64.abs().amax(1)
        # a row's sum passes through at most 16 + 10 + 16 additions
        close(mean, m64, 50 * U32 * big, "mean")
        er = 200 * U32 * (1 + big * r64)  # of rstd, relative: from the mean's error and the squares' sum
        close(rstd, r64, er * r64, "rstd")
        exh = er[:, None] * (xh.abs() + 1) + 60 * U32 * (big * r64)[:, None]
        ref = xh * gm64 + bt64
        close(y, ref, u(t) * ref.abs() + exh * gm64.abs() + 4 * U32 * (ref.abs() + bt64.abs()) + 2.0 ** -25, "y")
        dx, dg, db = op.backward(dy, x, gm, mean, rstd)
        a = dy.double() * gm64
        ma, mx = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
        ref = (a - ma - xh * mx) * r64[:, None]
        mag = (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True)) * r64[:, None]
        slip = exh * (mx.abs() + (a.abs()).mean(1, keepdim=True) * (1 + xh.abs())) * r64[:, None]
        close(dx, ref, u(t) * ref.abs() + (60 * U32 + er[:, None]) * mag + slip + 2.0 ** -25, "dx")
        pt = F32 if gm is None else gm.dtype
        dy64 = dy.double()
        ref, mag = (dy64 * xh).sum(0), (dy64 * xh).abs().sum(0)
        extra = (dy64.abs() * exh).sum(0)
        close(dg, ref, u(pt) * ref.abs() + (n + 4) * U32 * mag + extra + 2.0 ** -25, "dgamma")
        ref, mag = dy64.sum(0), dy64.abs().sum(0)
        close(db, ref, u(pt) * ref.abs() + (n + 4) * U32 * mag + 2.0 ** -25, "dbeta")
        again = op.backward(dy, x, gm, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip((dx, dg, db), again))


def test_norm_of_constant_rows_and_large_offsets():
    op = tt.LayerNorm(300, eps=1e-5)
    x = torch.full((4, 300), 3.25, device=DEV)
    x[1] = 0
    x[2] = 1e4 + torch.randn(300, device=DEV, generator=gen(1))
    x[3] = -1e30
    y, mean, rstd = op.forward(x)
    assert (y[0] == 0).all() and (y[1] == 0).all() and (y[3] == 0).all()
    assert torch.allclose(rstd[:2], torch.full((2,), 1e-5 ** -0.5, device=DEV), rtol=4 * U32)
    x64 = x[2].double()
    r64 = float(1 / (x64.var(correction=0) + 1e-5).sqrt())
    # the mean is off by at most 50 u of 1e4, a shift of every value
    assert float((y[2].double() - (x64 - x64.mean()) * r64).abs().max()) <= 60 * U32 * 1e4 * r64 * 2
    dx, dg, db = op.backward(torch.ones_like(x), x, None, mean, rstd)
    assert torch.isfinite(dx).all() and (db == 4).all()


def test_norm_gradient_against_differences():
    n, D = 3, 24
    op = tt.LayerNorm(D, eps=1e-2)
    g = gen(9)
    x, dy, gamma = rows(g, n, D, F32), rows(g, n, D, F32), rows(g, 1, D, F32)[0].contiguous()
    y, mean, rstd = op.forward(x, gamma)
    dx, dg, _ = op.backward(dy, x, gamma, mean, rstd)

    def loss(xv, gv):
        c = xv.double() - xv.double().mean(1, keepdim=True)
        return float((dy.double() * c / (c.square().mean(1, keepdim=True) + 1e-2).sqrt() * gv.double()).sum())

    h = 2.0 ** -10
    for i in range(n):
        for j in range(0, D, 5):
            p, q = x.double(), x.double()
            p[i, j] += h
            q[i, j] -= h
            # central differences: third derivatives are below 10^2 here, h^2 / 6 of them
            assert abs((loss(p, gamma) - loss(q, gamma)) / (2 * h) - float(dx[i, j])) <= 1e2 * h * h + 1e-5
    for j in range(0, D, 5):
        p, q = gamma.double(), gamma.double()
        p[j] += h
        q[j] -= h
        assert abs((loss(x, p) - loss(x, q)) / (2 * h) - float(dg[j])) <= 1e-5


def test_norm_of_no_rows():
    op = tt.LayerNorm(20)
    x = torch.zeros((0, 20), device=DEV)
    y, mean, rstd = op.forward(x)
    dx, dg, db = op.backward(x, x, torch.ones(20, device=DEV), mean, rstd)
    assert y.shape == dx.shape == (0, 20) and (dg == 0).all() and (db == 0).all()


def test_norm_keeps_a_nan_in_its_row():
    op = tt.LayerNorm(96)
    x = rows(gen(2), 40, 96, BF16).clone()
    clean = op.forward(x)[0]
    x[7, 5] = float("nan")
    y = op.forward(x)[0]
    assert y[7].isnan().all() and torch.equal(y[:7], clean[:7]) and torch.equal(y[8:], clean[8:])


# --------------------------------------------------------------------- xent

XENT = [(1, 1, 1, 0), (1, 2, 3, 0), (2, 130, 64, 0), (5, 1000, 72, 1), (64, 129, 128, 64), (130, 257, 40, 0),
        (200, 5003, 96, 3), (129, 640, 520, 8), (300, 40000, 64, 0), (33, 700, 1030, 0), (260, 2048, 256, 0)]


def xent_inputs(n, V, D, t, gap, seed):
    g = gen(seed)
    h, w = rows(g, n, D, t, gap), rows(g, V, D, t, gap, 2.0 / math.sqrt(D))
    target = torch.randint(0, V, (n,), device=DEV, generator=g)
    grad = torch.rand(n, device=DEV, generator=g)
    return h, w, target, grad


def xent_reference(h, w, target, grad, ignore):
    h, w = h.double(), w.double()
    z = h @ w.t()
    lse = torch.logsumexp(z, 1)
    counts = target != ignore
    at = torch.where(counts, target, 0)
    loss = torch.where(counts, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    p = (z - lse[:, None]).exp()
    one = torch.zeros_like(p).scatter_(1, at[:, None], 1.0)
    d = (p - one) * (grad.double() * counts)[:, None]
    mag = (p + one) * (grad.double().abs() * counts)[:, None]
    return z, lse, loss, d, mag


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D,gap", XENT)
def test_xent_and_gradients(n, V, D, gap, t):
    print(f"[case] xent n={n} V={V} D={D} gap={gap} {t}", flush=True)
    h, w, target, grad = xent_inputs(n, V, D, t, gap, n + V)
    target[n // 2] = -100
    grad[n // 2] = float("nan")  # an ignored row's gradient is not read into anything
    z, lse, loss, d, mag = xent_reference(h, w, target, torch.nan_to_num(grad), -100)
    h64, w64 = h.double(), w.double()
    # logits: fp32 sums of D products (six for fp32 inputs, split to 2^-25)
    ez = ((6 * D if t == F32 else D) + 8) * U32 * (h64.abs() @ w64.abs().t()).amax(1)
    # exponentials: the argument's rounding and 2 ulp of the instruction; sums of a tile, of the tiles
    ex = U32 * (4 + 2 * (z - lse[:, None]).abs().amax(1))
    es = ez + ex + (200 + V / 1024) * U32
    x = tt.VocabCrossEntropy(V, D)
    got_loss, got_lse = x.forward(h, w, target)
    close(got_lse, lse, es + 4 * U32 * lse.abs(), "lse")
    close(got_loss, loss, es + ez + 4 * U32 * (lse.abs() + z.abs().amax(1)), "loss")
    assert got_loss[n // 2] == 0
    l2, s2, dh, dw = x.loss_and_grad(h, w, target, grad)
    assert torch.equal(l2, got_loss) and torch.equal(s2, got_lse)
    # d: its own rounding (bf16, or three terms) and the error of the exponent
    ed = ((u(BF16) if t == BF16 else 2.0 ** -23) + ez + es + ex)[:, None] * mag
    ref = d @ w64
    k = 6 if t == F32 else 1
    close(dh, ref, ed @ w64.abs() + k * (V + 8) * U32 * (mag @ w64.abs()) + u(t) * ref.abs(), "dh")
    ref = d.t() @ h64
    close(dw, ref, ed.t() @ h64.abs() + k * (n + 8) * U32 * (mag.t() @ h64.abs()) + u(t) * ref.abs(), "dw")
    assert (dh[n // 2] == 0).all()
    again = x.loss_and_grad(h, w, target, grad)
    assert torch.equal(again[2], dh) and torch.equal(again[3], dw)
    assert x.poll_error() == 0


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D,gap", [(1024, 33000, 1024, 0), (1100, 66000, 40, 0), (513, 20011, 600, 8)])
def test_xent_in_large_tiles(n, V, D, gap, t):
    # enough rows, vocabulary and columns for 256 x 256 tiles in every product,
    # for tiles taken in patches, and for sums split over compute units
    test_xent_and_gradients(n, V, D, gap, t)


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D,gap", [(1, 33, 64, 0), (129, 257, 65, 0), (300, 5000, 128, 0), (4100, 40, 100, 3),
                                       (70, 20011, 128, 8), (1000, 100, 1, 0), (257, 31, 64, 8), (33, 1, 127, 0),
                                       (2000, 9001, 63, 1)])
def test_xent_of_narrow_rows(n, V, D, gap, t):
    # up to 128 columns: one operand in registers, the other streamed 32 rows at
    # a step, in whole steps and not, once and in splits
    test_xent_and_gradients(n, V, D, gap, t)


@pytest.mark.parametrize("n", [1, 5, 31, 32, 33, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("V,D,gap", [(1, 5, 0), (127, 31, 3), (128, 32, 0), (257, 33, 1), (1000, 100, 0), (3001, 516, 4)])
def test_xent_scores_of_few_rows(n, V, D, gap):
    # fp32 rows up to 128 take the weight as it is, more are split into terms
    h, w, target, grad = xent_inputs(n, V, D, F32, gap, n + V + D)
    z, lse, loss, _, _ = xent_reference(h, w, target, grad, -100)
    ez = (6 * D + 8) * U32 * (h.double().abs() @ w.double().abs().t()).amax(1)
    es = ez + U32 * (204 + V / 1024 + 2 * (z - lse[:, None]).abs().amax(1))
    x = tt.VocabCrossEntropy(V, D)
    got_loss, got_lse = x.forward(h, w, target)
    close(got_lse, lse, es + 4 * U32 * lse.abs(), "lse")
    close(got_loss, loss, es + ez + 4 * U32 * (lse.abs() + z.abs().amax(1)), "loss")
    assert x.poll_error() == 0


@pytest.mark.parametrize("t", [F32, BF16])
def test_xent_ignores_what_ignored_rows_hold(t):
    n, V, D = 70, 900, 96
    h, w, target, grad = xent_inputs(n, V, D, t, 0, 15)
    h = h.clone()
    x = tt.VocabCrossEntropy(V, D)
    target[5], target[40] = -100, -100
    ref = x.loss_and_grad(h, w, target, grad)
    h[5, 3], h[5, 7], h[40, 95] = float("nan"), float("inf"), float("-inf")
    got = x.loss_and_grad(h, w, target, grad)
    assert got[0][5] == 0 and got[0][40] == 0
    keep = target != -100
    assert all(torch.equal(p[keep], q[keep]) for p, q in zip(got[:3], ref[:3]))
    assert (got[2][~keep] == 0).all()
    # the two rows' zeros, instead of finite values, meet zero gradients: the same sums
    assert torch.equal(got[3], ref[3])


@pytest.mark.parametrize("t", [F32, BF16])
def test_xent_of_rows_of_very_different_size(t):
    # a hidden row 2^40 times another: each row's gradient keeps its own precision
    n, V, D = 64, 500, 64
    h, w, target, grad = xent_inputs(n, V, D, t, 0, 16)
    size = torch.exp2(torch.linspace(-40, 0, n, device=DEV))[:, None]
    h = (h * size).to(t)
    grad = torch.full_like(grad, 1.0 / n)
    z, lse, loss, d, mag = xent_reference(h, w, target, grad, -100)
    x = tt.VocabCrossEntropy(V, D)
    got = x.loss_and_grad(h, w, target, grad)
    ez = (6 * D + 8) * U32 * (h.double().abs() @ w.double().abs().t()).amax(1)
    es = ez + 210 * U32
    close(got[1], lse, es + 4 * U32 * lse.abs(), "lse")
    close(got[0], loss, es + ez + 4 * U32 * (lse.abs() + z.abs().amax(1)), "loss")
    # d's rounding (two fp16 terms, 2^-22, or bf16's)
    ed = ((u(BF16) if t == BF16 else 2.0 ** -21) + 2 * ez + 220 * U32)[:, None] * mag
    ref = d @ w.double()
    close(got[2], ref, ed @ w.double().abs() + 6 * (V + 8) * U32 * (mag @ w.double().abs()) + u(t) * ref.abs(), "dh")
    # the hidden values' own floor beside the largest row (fp32 inputs): 2^-38 of it
    ref = d.t() @ h.double()
    ed = ((u(BF16) if t == BF16 else 2.0 ** -21) + 2 * ez + 220 * U32)[:, None] * mag
    close(got[3], ref, ed.t() @ h.double().abs() + 6 * (n + 8) * U32 * (mag.t() @ h.double().abs())
          + u(t) * ref.abs() + 2.0 ** -38 * h.double().abs().max() * mag.sum(0)[:, None], "dw")


@pytest.mark.parametrize("t", [F32, BF16])
def test_xent_in_small_pieces_is_the_same(t):
    n, V, D = 150, 3000, 80
    h, w, target, grad = xent_inputs(n, V, D, t, 0, 5)
    whole = tt.VocabCrossEntropy(V, D)
    ref = whole.loss_and_grad(h, w, target, grad)
    least = whole._need(n, 0 if t == F32 else 1, True, "test")
    small = tt.VocabCrossEntropy(V, D, max_workspace=1)
    with pytest.raises(tt.TTEmbError) as e:
        small.loss_and_grad(h, w, target, grad)
    assert e.value.status == tt.TT_EMB_ERR_WORKSPACE
    need = int(str(e.value).split("at least ")[1].split()[0])
    assert need < least
    small = tt.VocabCrossEntropy(V, D, max_workspace=need)
    got = small.loss_and_grad(h, w, target, grad)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[3], ref[3])
    # dH is summed piece by piece: another order of the same sum
    d = xent_reference(h, w, target, grad, -100)[4]
    bound = 12 * (V + 8) * U32 * (d @ w.double().abs()) + 2 * u(t) * ref[2].double().abs()
    close(got[2], ref[2], bound, "dh")


def test_xent_of_peaked_rows_stays_finite():
    # logits near +-1e4: every exponential but the largest underflows
    n, V, D = 40, 600, 64
    for t in (F32, BF16):
        h, w, target, grad = xent_inputs(n, V, D, t, 0, 6)
        h = h * 2000
        z, lse, loss, d, _ = xent_reference(h, w, target, grad, -100)
        x = tt.VocabCrossEntropy(V, D)
        got = x.loss_and_grad(h, w, target, grad)
        ez = (8 * D) * U32 * (h.double().abs() @ w.double().abs().t()).amax(1)
        close(got[1], lse, 2 * ez + 4 * U32 * lse.abs(), "lse")
        close(got[0], loss, 4 * ez + 4 * U32 * lse.abs(), "loss")
        assert torch.isfinite(got[2]).all() and torch.isfinite(got[3]).all()


def test_xent_all_ignored_and_targets_out_of_range():
    n, V, D = 20, 300, 64
    h, w, target, grad = xent_inputs(n, V, D, BF16, 0, 7)
    x = tt.VocabCrossEntropy(V, D, ignore_index=-7)
    loss, lse, dh, dw = x.loss_and_grad(h, w, torch.full_like(target, -7), grad)
    assert (loss == 0).all() and (dh == 0).all() and (dw == 0).all() and torch.isfinite(lse).all()
    assert x.poll_error() == 0
    clean = target.clone()
    clean[4] = -7
    ref = x.loss_and_grad(h, w, clean, grad)
    for bad in (-1, V, 2 ** 40, -2 ** 60):
        target[4] = bad
        got = x.loss_and_grad(h, w, target, grad)
        assert x.poll_error() == tt.TT_EMB_ERR_INDEX
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
        assert x.poll_error() == 0


def test_xent_of_no_rows():
    x = tt.VocabCrossEntropy(100, 48)
    for t in (F32, BF16):
        h, w = torch.zeros((0, 48), device=DEV, dtype=t), torch.ones((100, 48), device=DEV, dtype=t)
        none = torch.zeros(0, dtype=torch.int64, device=DEV)
        loss, lse, dh, dw = x.loss_and_grad(h, w, none, torch.zeros(0, device=DEV))
        assert loss.numel() == lse.numel() == dh.numel() == 0 and (dw == 0).all()


def test_xent_gradient_against_differences():
    n, V, D = 3, 9, 6
    h, w, target, grad = xent_inputs(n, V, D, F32, 0, 8)
    _, _, dh, dw = tt.VocabCrossEntropy(V, D).loss_and_grad(h, w, target, grad)

    def total(hv, wv):
        return float((xent_reference(hv, wv, target, grad, -100)[2] * grad.double()).sum())

    step = 2.0 ** -10
    for a, da in ((h, dh), (w, dw)):
        for i in range(a.shape[0]):
            for j in range(a.shape[1]):
                p, q = a.double(), a.double()
                p[i, j] += step
                q[i, j] -= step
                hi, lo = (total(p, w), total(q, w)) if a is h else (total(h, p), total(h, q))
                # third derivatives of lse by one entry are below 10^2 here
                assert abs((hi - lo) / (2 * step) - float(da[i, j])) <= 1e2 * step * step + 1e-5


# -------------------------------------------------------------------- adamw

def adamw_reference(p, g, m, v, step, lr=1e-2, b1=0.9, b2=0.99, eps=1e-6, wd=0.1):
    p, g, m, v = (x.double() for x in (p, g, m, v))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    up = (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + eps)
    return p * (1 - lr * wd) - lr * up, m, v, lr * up.abs()


SIZES = [[1], [255, 256, 257], [3, 4096, 1, 5000, 0, 7], [70001], [17] * 200]


@pytest.mark.parametrize("gt", TYPES)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_adamw_with_states_in_32_bits(sizes, gt):
    g = gen(len(sizes))
    params = [torch.randn(s, device=DEV, generator=g) for s in sizes]
    copies = [torch.zeros(s, device=DEV, dtype=BF16) for s in sizes]
    opt = tt.AdamW(params, lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1, copies=copies)
    at = [0]
    for s in sizes:
        at.append(at[-1] + (s + 255) // 256 * 256)
    for step in (1, 2, 3):
        grads = [torch.randn(s, device=DEV, generator=g).to(gt) for s in sizes]
        before = [(p.clone(), opt.exp_avg[a:a + s].clone(), opt.exp_avg_sq[a:a + s].clone())
                  for p, a, s in zip(params, at, sizes)]
        opt.step(grads)
        for (p0, m0, v0), p, c, gr, a, s in zip(before, params, copies, grads, at, sizes):
            rp, rm, rv, up = adamw_reference(p0, gr, m0, v0, step)
            m, v = opt.exp_avg[a:a + s], opt.exp_avg_sq[a:a + s]
            close(m, rm, 4 * U32 * (m0.double().abs() + gr.double().abs()), "m")
            close(v, rv, 6 * U32 * rv, "v")
            # m's error is relative to its terms, divided by the root like m itself
            slip = 8 * U32 * 1e-2 * (m0.double().abs() + gr.double().abs()) / (1 - 0.9 ** step) / (
                (rv / (1 - 0.99 ** step)).sqrt() + 1e-6)
            close(p, rp, 4 * U32 * p0.double().abs() + 16 * U32 * up + slip, "p")
            assert torch.equal(c, p.to(BF16))
    assert opt.steps == 3


def e4m3(code, scale):
    return code.double() * scale.double().repeat_interleave(256)


@pytest.mark.parametrize("sizes", [[1], [256, 300, 5], [70001], [17] * 100], ids=lambda s: f"{len(s)}x{s[0]}")
def test_adamw_with_states_in_8_bits(sizes):
    g = gen(len(sizes))
    params = [torch.randn(s, device=DEV, generator=g) for s in sizes]
    opt = tt.AdamW(params, lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1, state_bits=8, seed=11)
    flat = sum((s + 255) // 256 * 256 for s in sizes)
    assert opt.exp_avg.numel() == flat and opt.exp_avg_scale.numel() == flat // 256

    def pad(ts):
        return torch.cat([torch.cat([x.reshape(-1).float(),
                                     torch.zeros(-x.numel() % 256, device=DEV)]) for x in ts])

    for step in (1, 2, 3, 4):
        grads = [torch.randn(s, device=DEV, generator=g) * 10.0 ** float(torch.randn((), generator=torch.Generator().manual_seed(step)))
                 for s in sizes]
        m0, v0 = e4m3(opt.exp_avg, opt.exp_avg_scale), e4m3(opt.exp_avg_sq, opt.exp_avg_sq_scale)
        p0 = pad(params)
        opt.step(grads)
        gr = pad(grads)
        rp, rm, rv, up = adamw_reference(p0, gr, m0, v0, step)
        m, v = e4m3(opt.exp_avg, opt.exp_avg_scale), e4m3(opt.exp_avg_sq, opt.exp_avg_sq_scale)
        sm, sv = (x.double().repeat_interleave(256) for x in (opt.exp_avg_scale, opt.exp_avg_sq_scale))
        # each value is one of its two neighbours: within a spacing (2^-3 and
        # 2^-2 of the value, or the spacing of the smallest values)
        near = 1 + 1e-5
        close(m, rm, near * torch.maximum(rm.abs() / 8, sm * 2.0 ** -9) + 8 * U32 * (m0.abs() + gr.double().abs()), "m")
        close(v, rv, near * torch.maximum(rv / 4, sv * 2.0 ** -16) + 8 * U32 * rv, "v")
        assert ((v > 0) | (rv == 0)).all()
        slip = 8 * U32 * 1e-2 * (m0.abs() + gr.double().abs()) / (1 - 0.9 ** step) / (
            (rv / (1 - 0.99 ** step)).sqrt() + 1e-6)
        close(pad(params), rp, 4 * U32 * p0.double().abs() + 16 * U32 * up + slip, "p")
        top = rm.view(-1, 256).abs().amax(1)
        close(opt.exp_avg_scale, torch.clamp(top, min=2.0 ** -100) / 448, 1e-5 * top / 448 + 2.0 ** -130, "scale")


def test_adamw_rounds_at_random_without_bias():
    # one value far below the block's largest, again and again with new steps:
    # the mean of the stored values is the value
    n = 256 * 512
    p = torch.zeros(n, device=DEV)
    grad = torch.full((n,), 0.3, device=DEV)
    grad[::256] = 100.0
    opt = tt.AdamW([p], betas=(0.9, 0.999), state_bits=8, seed=3)
    got = []
    for _ in range(16):
        opt.load_state(torch.zeros_like(opt.exp_avg.view(torch.uint8)).view(torch.float8_e4m3fn),
                       torch.zeros_like(opt.exp_avg_sq.view(torch.uint8)).view(torch.float8_e5m2),
                       len(got), torch.zeros_like(opt.exp_avg_scale), torch.zeros_like(opt.exp_avg_sq_scale))
        opt.step([grad])
        got.append((e4m3(opt.exp_avg, opt.exp_avg_scale), e4m3(opt.exp_avg_sq, opt.exp_avg_sq_scale)))
    at = torch.arange(n, device=DEV) % 256 != 0
    for k, true in ((0, 0.03), (1, 0.001 * 0.09)):
        x = torch.stack([q[k][at] for q in got])
        spacing = true / 4 if k else true / 8
        # mean of 2e6 independent values of a spread below half a spacing, five sigma; 2^-16 of a
        # spacing is what 16 random bits cannot tell
        assert abs(float(x.mean()) - true) <= spacing * (5 * 0.5 / math.sqrt(x.numel()) + 2.0 ** -15) + 1e-6 * true
        assert len(torch.unique(x)) == 2


def test_adamw_is_reproducible_and_depends_on_seed_and_step():
    def go(seed, start):
        g = gen(4)
        p = torch.randn(5000, device=DEV, generator=g)
        opt = tt.AdamW([p], state_bits=8, seed=seed)
        opt.steps = start
        opt.step([torch.randn(5000, device=DEV, generator=g)])
        return opt.exp_avg.view(torch.uint8).clone()

    assert torch.equal(go(1, 0), go(1, 0))
    assert not torch.equal(go(1, 0), go(2, 0)) and not torch.equal(go(1, 0), go(1, 5))


def test_adamw_of_gradients_with_nan_and_infinity():
    for bits in (32, 8):
        p = torch.ones(600, device=DEV)
        opt = tt.AdamW([p], state_bits=bits)
        grad = torch.ones(600, device=DEV)
        grad[300], grad[20] = float("nan"), float("inf")
        opt.step([grad])
        assert p[300].isnan() and torch.isfinite(p[512:]).all() and torch.isfinite(p[301:400]).all()
        m = opt.exp_avg.float()
        if bits == 8:
            m = m * opt.exp_avg_scale.repeat_interleave(256)
            assert m[256:512].isnan().all() and m[:256].isnan().all() and torch.isfinite(m[512:]).all()
        else:
            assert m[300].isnan() and torch.isfinite(m[301:]).all()


def test_adamw_of_zero_gradients_decays_only():
    for bits in (32, 8):
        p = torch.ones(300, device=DEV)
        opt = tt.AdamW([p], lr=0.1, weight_decay=0.5, state_bits=bits)
        opt.step([torch.zeros(300, device=DEV)])
        assert torch.allclose(p, torch.full_like(p, 0.95), rtol=2 * U32) and (opt.exp_avg.float() == 0).all()


def test_adamw_takes_tensors_at_odd_places():
    # views of a flat buffer that begin at any element
    g = gen(6)
    flat, grad = torch.randn(3000, device=DEV, generator=g), torch.randn(3000, device=DEV, generator=g)
    cut = [(1, 300), (302, 1), (305, 1025), (1333, 1600)]
    own = [flat[a:a + n].clone() for a, n in cut]
    views = [flat[a:a + n] for a, n in cut]
    rest = flat.clone()
    x, y = tt.AdamW(views), tt.AdamW(own)
    for _ in range(2):
        x.step([grad[a:a + n] for a, n in cut])
        y.step([grad[a:a + n].clone() for a, n in cut])
    assert all(torch.equal(p, q) for p, q in zip(views, own))
    for a, n in cut:
        rest[a:a + n] = flat[a:a + n]
    assert torch.equal(rest, flat)


# ------------------------------------------------- streams, graphs, together

def small_step(ops, w, tok, gamma, target, grad, stream=None):
    e, ln, xe = ops
    x = e.forward(w, tok, stream=stream)
    y, mean, rstd = ln.forward(x, gamma, None, stream=stream)
    loss, lse, dy, dw = xe.loss_and_grad(y, w, target, grad, stream=stream)
    dx, dg, _ = ln.backward(dy, x, gamma, mean, rstd, stream=stream)
    e.backward(dx, tok, grad_weight=dw, accumulate=True, stream=stream)
    return loss, dw, dg


def small_inputs(t=BF16):
    V, D, n = 700, 128, 96
    g = gen(12)
    w = rows(g, V, D, t, 0, 0.1)
    tok, target = (torch.randint(0, V, (n,), device=DEV, generator=g) for _ in range(2))
    gamma = torch.ones(D, device=DEV)
    ops = tt.TokenEmbedding(V, D, scale=math.sqrt(D), padding_idx=0), tt.LayerNorm(D), tt.VocabCrossEntropy(V, D)
    return ops, w, tok, gamma, target, torch.full((n,), 1.0 / n, device=DEV)


def test_operators_run_on_the_stream_they_are_given():
    args = small_inputs()
    ref = small_step(*args)
    torch.cuda.synchronize()
    for make in (lambda s: s, lambda s: s.cuda_stream):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = small_step(*args, stream=make(s))
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_operators_in_a_captured_graph():
    ops, w, tok, gamma, target, grad = small_inputs(F32)
    opt = tt.AdamW([w, gamma], lr=1e-2, state_bits=8)

    def step():
        loss, dw, dg = small_step(ops, w, tok, gamma, target, grad)
        opt.step([dw, dg])
        return loss

    keep = [x.clone() for x in (w, gamma, opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8),
                                opt.exp_avg_scale, opt.exp_avg_sq_scale)]

    def reset():
        for x, k in zip((w, gamma, opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8),
                         opt.exp_avg_scale, opt.exp_avg_sq_scale), keep):
            x.copy_(k)
        opt.steps = 0

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = step()
    for _ in range(3):  # the captured step is step 1 every time
        losses = []
        reset()
        eager = step().clone()
        after = w.clone()
        reset()
        graph.replay()
        torch.cuda.synchronize()
        losses.append(captured.clone())
        assert torch.equal(losses[0], eager) and torch.equal(w, after)
        assert all(op.poll_error() == 0 for op in (ops[0], ops[2]))


def test_a_few_steps_lower_the_loss():
    ops, w, tok, gamma, target, grad = small_inputs(F32)
    opt = tt.AdamW([w, gamma], lr=1e-2, weight_decay=0.0)
    losses = []
    for _ in range(30):
        loss, dw, dg = small_step(ops, w, tok, gamma, target, grad)
        opt.step([dw, dg])
        losses.append(float(loss.mean()))
    assert losses[-1] < 0.5 * losses[0]
