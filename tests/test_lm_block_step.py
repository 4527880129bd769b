"""A block and its training step as they are used together: norm, gated
feed-forward block, gate and residual, loss, gradients, their bound and AdamW;
alone in fp32 and bf16, in a captured graph, and in the example model."""

import math

import pytest
import test_lm_example as ex
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

pytestmark = pytest.mark.gpu
F32, BF16, DEV = ops.F32, ops.BF16, ops.DEV


class Model:
    """Two blocks over rows of D elements, scored against a vocabulary."""

    def __init__(self, t, D=96, F=160, V=500, seed=0):
        g = ops.gen(seed)
        self.t, self.D = t, D
        rows = lambda n, m, std: ops.rows(g, n, m, t, 0, std)  # noqa: E731
        self.w = {"table": rows(V, D, 1.0 / math.sqrt(D))}
        for k in (0, 1):
            self.w[f"in{k}"], self.w[f"out{k}"] = rows(2 * F, D, 1 / math.sqrt(D)), rows(D, F, 1 / math.sqrt(F))
            for name in ("gate", "gamma", "post_gamma"):
                self.w[f"{name}{k}"] = (0.5 + torch.rand(D, device=DEV, generator=g)).to(t)
        self.gamma = torch.ones(D, device=DEV)
        self.first = tt.LayerNorm(D)
        self.feed = [tt.GatedFeedForward(D, F, activation=a) for a in ("silu", "gelu_tanh")]
        self.between = [tt.BlockNorm(D, post=True, block_scale=0.5) for _ in (0, 1)]
        self.loss = tt.VocabCrossEntropy(V, D)

    def _block(self, k):
        return {n: self.w[f"{n}{k}"] for n in ("gate", "gamma", "post_gamma")}

    def grads(self, x, target, grad_loss):
        y, mean, rstd = self.first.forward(x, self.gamma)
        h, kept = x, []
        for k in (0, 1):
            f, pre = self.feed[k].forward(y, self.w[f"in{k}"], self.w[f"out{k}"], keep=True)
            y2, h2, stats = self.between[k].forward(f, h, **self._block(k))
            kept.append((y, h, f, pre, stats))
            y, h = y2, h2
        loss, _, dy, dtable = self.loss.loss_and_grad(y, self.w["table"], target, grad_loss)
        out, dh = {"table": dtable}, None
        for k in (1, 0):
            y, h, f, pre, stats = kept[k]
            df, dh, dgate, dgamma, _, dpost, _ = self.between[k].backward(dy, dh, f, h, stats, **self._block(k))
            dy, out[f"in{k}"], out[f"out{k}"] = self.feed[k].backward(df, y, pre, self.w[f"in{k}"], self.w[f"out{k}"])
            out[f"gate{k}"], out[f"gamma{k}"], out[f"post_gamma{k}"] = dgate, dgamma, dpost
        dx = self.first.backward(dy, x, self.gamma, mean, rstd)[0]
        return loss, {"x": dx + dh, **out}

    def grads64(self, x, target, grad_loss):
        leaves = {"x": x, **self.w}
        leaves = {k: v.double().requires_grad_() for k, v in leaves.items()}
        rms = lambda v: v * (v.square().mean(1, keepdim=True) + 1e-5).rsqrt()  # noqa: E731
        h = leaves["x"]
        y = torch.nn.functional.layer_norm(h, (self.D,))
        for k, act in ((0, torch.nn.functional.silu), (1, lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
            g, u = (y @ leaves[f"in{k}"].t()).chunk(2, 1)
            f = (act(g) * u) @ leaves[f"out{k}"].t()
            h = h + 0.5 * leaves[f"gate{k}"] * (rms(f) * leaves[f"post_gamma{k}"])
            y = rms(h) * leaves[f"gamma{k}"]
        loss = torch.nn.functional.cross_entropy(y @ leaves["table"].t(), target, reduction="none")
        (loss * grad_loss.double()).sum().backward()
        return loss.detach(), {k: v.grad for k, v in leaves.items()}


def inputs(t, n, D=96, V=500, seed=1):
    g = ops.gen(seed)
    return (ops.rows(g, n, D, t), torch.randint(0, V, (n,), device=DEV, generator=g),
            torch.rand(n, device=DEV, generator=g) / n)


# fp32: some forty sums of at most 500 terms in a row, each to 2^-22 of its terms:
# 1e-4 of the largest value leaves a factor of ten.  bf16: activations and their
# gradients are rounded to 2^-9 some fifteen times on the way down and up again,
# and add up as independent errors do: 15^(1/2) x 2^-9 = 0.8 % of the root mean
# square; three times that.
@pytest.mark.parametrize("t,n", [(F32, 40), (F32, 300), (BF16, 40), (BF16, 300)])
def test_gradients_of_two_blocks(t, n):
    m, args = Model(t), inputs(t, n)
    loss, got = m.grads(*args)
    ref_loss, ref = m.grads64(*args)
    assert set(got) == set(ref)
    scale = 1e-4 if t == F32 else 0.024
    assert float((loss.double() - ref_loss).square().mean().sqrt()) <= scale * float(ref_loss.square().mean().sqrt())
    for k in ref:
        assert got[k].dtype == t and got[k].shape == ref[k].shape, k
        off = float((got[k].double() - ref[k]).square().mean().sqrt())
        assert off <= scale * float(ref[k].square().mean().sqrt()), k


def test_a_step_in_a_graph():
    # forward, backward, bound and update, captured once and replayed with new inputs
    t, n = BF16, 200
    m = Model(t)
    names = list(m.w)
    master = {k: v.float() for k, v in m.w.items()}
    opt = tt.AdamW([master[k] for k in names], lr=1e-3, copies=[m.w[k] for k in names])
    clip = tt.GradientClip(0.05)
    x, target, grad_loss = inputs(t, n)
    start = {k: v.clone() for k, v in master.items()}

    def gradients():
        _, g = m.grads(x, target, grad_loss)
        g = [g[k] for k in names]
        return g, clip.norm(g)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gradients()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g, (norm, factor) = gradients()

    def run(step):
        for k in names:
            master[k].copy_(start[k])
            m.w[k].copy_(start[k])
        opt.exp_avg.zero_(), opt.exp_avg_sq.zero_()
        opt.steps = 0
        seen = []
        for seed in (5, 6, 7):
            for a, b in zip((x, target, grad_loss), inputs(t, n, seed=seed)):
                a.copy_(b)
            torch.cuda.synchronize()
            grads, bound = step()
            opt.step(grads, grad_scale=bound[1])
            torch.cuda.synchronize()
            seen += [float(bound[0]), float(bound[1])] + [master[k].clone() for k in names]
        return seen

    def replay():
        graph.replay()
        torch.cuda.synchronize()
        return g, (norm, factor)

    eager, captured = run(gradients), run(replay)
    for a, b in zip(eager, captured):
        assert torch.equal(a, b) if torch.is_tensor(a) else a == b
    assert 0 < eager[1] < 1 and eager[0] > 0.05  # the bound held the gradients
    for op in [m.first, m.loss, clip, *m.feed, *m.between]:
        assert op.poll_error() == 0


def test_the_example_with_a_block_takes_the_gradient_of_its_loss():
    e = ex.example()
    model = e.NextToken(hidden=48, clip=1e-3)
    assert len(model.params) == 13
    context, target = next(e.batches(model, 64))
    before, taken = [p.clone() for p in model.params], []
    model.opt.step = lambda gs, grad_scale: taken.extend([list(gs), grad_scale])
    loss = model.step(context, target)
    model.check()
    assert all(torch.equal(p, q) for p, q in zip(before, model.params))
    leaves = [p.double().requires_grad_() for p in before]
    (c0, c1, c2), weight, gamma, beta, w_in, w_out = leaves[:3], *leaves[3:8]
    gate, g2, b2, pg, pb = leaves[8:]
    t = context.reshape(-1)
    i0, i1, i2 = t // 100, t // 10 % 10, t % 10
    rows = torch.einsum("nap,npbq,nqc->nabc", c0[i0][:, 0], c1[i1], c2[i2][..., 0]).reshape(len(t), -1)
    x = rows.view(64, -1, model.D).sum(1) + math.sqrt(model.D) * weight[context[:, -1]]
    norm = lambda v, a, b: torch.nn.functional.layer_norm(v, (model.D,), a, b, 1e-5)  # noqa: E731
    g, u = (norm(x, gamma, beta) @ w_in.t()).chunk(2, 1)
    f = (torch.nn.functional.silu(g) * u) @ w_out.t()
    y = norm(x + gate * norm(f, pg, pb), g2, b2)
    ref = torch.nn.functional.cross_entropy(y @ weight.t(), target, ignore_index=e.IGNORE, reduction="none")
    (ref.sum() / (target != e.IGNORE).sum()).backward()
    assert float((loss.double() - ref.detach()).abs().max()) <= 1e-4
    grads, factor = taken
    assert len(grads) == len(leaves)
    for k, (a, leaf) in enumerate(zip(grads, leaves)):
        # fp32 sums of up to 64 x 1000 terms, each to 2^-22, through three norms
        assert float((a.double() - leaf.grad).abs().max()) <= 2e-4 * float(leaf.grad.abs().max()), k
    size = math.sqrt(sum(float(leaf.grad.square().sum()) for leaf in leaves))
    assert abs(float(factor) - 1e-3 / size) <= 1e-3 * 1e-3 / size


@pytest.mark.parametrize("bits", [32, 8])
def test_the_example_runs_with_a_block_and_a_bound(bits):
    first, last = ex.example().train(5, bits, B=512, hidden=100, clip=0.5)
    assert math.isfinite(first) and math.isfinite(last)
