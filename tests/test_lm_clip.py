"""The global norm of the gradients of many tensors, their scaling to a bound,
and the AdamW step that takes the factor, against plain 64-bit forms.

Tolerances: N and the factor are fp64 results rounded to fp32 (2^-24, half a
step; the fp64 sum of k squares is off by at most k 2^-53).  A scaled gradient
is the product with the rounded factor (2^-24), rounded to fp32 (2^-24) and to
its type (eps / 2, or half of the smallest fp16 step)."""

import ctypes as C
import math

import pytest
import test_lm_abi as abi
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

F32, BF16, F16, U32, DEV = ops.F32, ops.BF16, ops.F16, ops.U32, ops.DEV
ARG, WS, UNSUPPORTED = abi.ARG, abi.WS, abi.UNSUPPORTED
INF, NAN = float("inf"), float("nan")


# ----------------------------------------------------------------- refusals

def clip(name="tt_emb_clip_scale", **bad):
    two = C.c_void_p * 2
    good = dict(count=2, grads=two(abi.P, abi.Q), dtypes=(C.c_int32 * 2)(0, 1), numel=(C.c_int64 * 2)(10, 7),
                max_norm=1.0, eps=1e-6, norm=abi.R, factor=abi.R + 4, ws=abi.W, ws_bytes=255, stream=None)
    return abi.call(name, good, **bad)


@pytest.mark.parametrize("name", ["tt_emb_clip_scale", "tt_emb_clip_norm"])
def test_entry_points_refuse(name):
    two, i64, i32 = C.c_void_p * 2, C.c_int64 * 2, C.c_int32 * 2
    for bad in (dict(count=-1), dict(grads=None), dict(dtypes=None), dict(numel=None), dict(numel=i64(-1, 5)),
                dict(grads=two(abi.P, None)), dict(grads=two(abi.P + 2, abi.Q)), dict(grads=two(abi.P, abi.Q + 1)),
                dict(dtypes=i32(0, 3)), dict(dtypes=i32(-1, 0)), dict(max_norm=-1.0), dict(max_norm=NAN),
                dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF), dict(norm=abi.R + 2), dict(factor=abi.R + 1)):
        assert clip(name, **bad) == ARG, bad
    for bad in (dict(), dict(ws=None), dict(ws=abi.W + 64, ws_bytes=4096), dict(count=0)):
        assert clip(name, **bad) == WS, bad  # (the good call has a byte too few)
    assert clip(name, numel=i64(2 ** 62, 2 ** 62)) == UNSUPPORTED
    assert clip(name, numel=i64(10, 0), grads=two(abi.P, None)) == WS  # nothing is read of an empty tensor


def test_tensors_that_share_memory_are_refused():
    two, i64 = C.c_void_p * 2, C.c_int64 * 2
    for q in (abi.P, abi.P + 4, abi.P + 36, abi.P - 12):
        assert clip(grads=two(abi.P, q)) == ARG, q
        assert clip("tt_emb_clip_norm", grads=two(abi.P, q)) == WS
    for q in (abi.P + 40, abi.P - 14):
        assert clip(grads=two(abi.P, q)) == WS, q
    assert clip(grads=two(abi.P, abi.P), numel=i64(10, 0)) == WS


def test_sizes():
    L, out = tt.lib(), C.c_size_t()
    numel = (C.c_int64 * 3)(1, 0, 5000)
    assert L.tt_emb_clip_workspace_size(3, numel, C.byref(out)) == 0 and out.value == 512
    assert L.tt_emb_clip_workspace_size(0, None, C.byref(out)) == 0 and out.value == 256
    assert L.tt_emb_clip_workspace_size(3, numel, None) == ARG
    assert L.tt_emb_clip_workspace_size(3, None, C.byref(out)) == ARG


def test_binding_refuses():
    for bad in (dict(max_norm=-1.0), dict(max_norm=NAN), dict(max_norm=1.0, eps=-1.0), dict(max_norm=1.0, eps=INF)):
        abi.refused(tt.GradientClip, **bad, msg="max_norm")
    c = tt.GradientClip(1.0)
    for f in (c.norm, c.clip):
        abi.refused(f, [], msg="no gradients")
        abi.refused(f, [torch.zeros(4)], msg="GPU")
        abi.refused(f, [None], msg="torch tensor")
        abi.refused(f, [torch.zeros(4).double()], msg="dtype")
        abi.refused(f, [torch.zeros(4, 4).t()[1:]], msg="contiguous")


def test_adamw_refuses_a_scale_it_would_misread():
    one = C.c_void_p * 1
    good = dict(count=1, params=one(abi.P), grads=one(abi.Q), gdt=0, scale=abi.R, copies=None,
                numel=(C.c_int64 * 1)(10), m=abi.R, v=abi.R, ms=None, vs=None, bits=32, lr=1e-3, b1=0.9, b2=0.99,
                eps=1e-8, wd=0.0, step=0, seed=0, stream=None)
    assert abi.call("tt_emb_adamw_update_scaled", good, step=1, scale=abi.R + 2) == ARG
    assert abi.call("tt_emb_adamw_update_scaled", good) == ARG  # step 0
    assert abi.call("tt_emb_adamw_update_scaled", good, count=0, step=1) == tt.TT_EMB_OK


# ------------------------------------------------------------------ results

SIZES = [[1], [0, 1, 0], [7, 5, 3], [4095], [4096], [4097], [16384, 1], [16385], [20000, 3, 4097], [5] * 159,
         [33] * 160, [100] * 161, [4096] * 161, [3, 70001] * 200, [9_000_001, 12, 500_000]]


def grads_of(sizes, kinds, seed, std=1.0):
    """Tensors of the sizes, at every alignment that their type allows."""
    g, out = ops.gen(seed), []
    for i, (n, k) in enumerate(zip(sizes, kinds)):
        at = i % 5
        flat = torch.full((n + at + 1,), NAN, device=DEV, dtype=k)  # what lies around is neither read nor written
        flat[at:at + n] = (std * torch.randn(n, device=DEV, generator=g)).to(k)
        out.append(flat[at:at + n])
    return out


def norm_of(grads):
    return math.sqrt(sum(float(x.double().square().sum()) for x in grads))


def check_scaled(got, before, factor, what):
    for i, (x, b) in enumerate(zip(got, before)):
        ref = b.double() * factor
        bound = ref.abs() * (ops.u(x.dtype) + 2 * U32) + (2.0 ** -25 if x.dtype == F16 else 2.0 ** -134)
        if x.numel():
            ops.close(x, ref, bound, f"{what} {i}")


@pytest.mark.gpu
@pytest.mark.parametrize("kinds", [[F32], [BF16], [F16], [F32, BF16, F16]], ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_scaling(sizes, kinds):
    print(f"[case] clip {len(sizes)} tensors of up to {max(sizes)} {kinds}", flush=True)
    grads = grads_of(sizes, kinds * len(sizes), len(sizes) + max(sizes))
    before = [x.clone() for x in grads]
    ref = norm_of(grads)
    c = tt.GradientClip(0.25 * ref)
    n, f = c.norm(grads)
    assert n.shape == f.shape == () and n.dtype == f.dtype == F32
    want = 0.25 * ref / (ref + 1e-6)
    assert abs(float(n) - ref) <= ref * (U32 + 2.0 ** -40)
    assert abs(float(f) - want) <= want * (U32 + 2.0 ** -40)
    assert all(torch.equal(x, b) for x, b in zip(grads, before))
    again = c.clip(grads)
    assert torch.equal(again, n)
    check_scaled(grads, before, float(f), "scaled")
    flat = [x.as_strided((x.numel() + 1,), (1,)) for x in grads]
    assert all(bool(y[-1].isnan()) for y in flat)
    # within the bound nothing is touched
    here = [x.clone() for x in grads]
    c.clip(grads, max_norm=0.25 * ref * 1.05)
    assert all(torch.equal(x, y) for x, y in zip(grads, here))
    assert c.poll_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[50, 3], [30000, 70000]], ids=["one", "many"])
def test_values_that_32_bits_cannot_square(sizes):
    # 1e30 and 1e-30: squares of 1e60 and 1e-60; subnormal values
    for size in (1e30, 1e-30, 1e-41):
        grads = grads_of(sizes, [F32, F32], 3, size)
        ref = norm_of(grads)
        n, f = tt.GradientClip(ref / 2, eps=0.0).norm(grads)
        assert abs(float(n) - ref) <= ref * 2 * U32 + 2.0 ** -150
        assert abs(float(f) - 0.5) <= 2 * U32
    # a norm past what fp32 holds: infinite there, the factor still right
    grads = [torch.full((sizes[0],), 3e38, device=DEV), torch.ones(sizes[1], device=DEV)]
    ref = 3e38 * math.sqrt(sizes[0])
    n, f = tt.GradientClip(1e38).norm(grads)
    assert float(n) == INF
    assert abs(float(f) - 1e38 / ref) <= 4 * U32  # (3e38 itself is off by 2^-24)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[50, 3], [30000, 70000]], ids=["one", "many"])
def test_edges_of_the_bound(sizes):
    zeros = [torch.zeros(n, device=DEV) for n in sizes]
    for bound, eps in ((0.0, 0.0), (1.0, 0.0), (1.0, 1e-6), (INF, 1e-6)):
        n, f = tt.GradientClip(bound, eps=eps).norm(zeros)
        assert float(n) == 0.0 and float(f) == 1.0
    assert float(tt.GradientClip(0.0).norm(zeros)[1]) == 0.0  # 0 / eps
    grads = grads_of(sizes, [F32, BF16], 1)
    keep = [x.clone() for x in grads]
    tt.GradientClip(INF).clip(grads)
    assert all(torch.equal(x, y) for x, y in zip(grads, keep))
    tt.GradientClip(0.0).clip(grads)
    assert all((x == 0).all() for x in grads)
    for bad in (INF, -INF, NAN):
        grads = [x.clone() for x in keep]
        grads[1][2] = bad
        n, f = tt.GradientClip(1.0).norm(grads)
        tt.GradientClip(1.0).clip(grads)
        if bad == bad:
            assert float(n) == INF and float(f) == 0.0
            assert (grads[0] == 0).all() and bool(grads[1][2].isnan()) and int(grads[1].isnan().sum()) == 1
        else:
            assert bool(n.isnan()) and bool(f.isnan()) and all(x.isnan().all() for x in grads)
    # nothing in any tensor
    n, f = tt.GradientClip(1.0).norm([torch.zeros(0, device=DEV)])
    assert float(n) == 0.0 and float(f) == 1.0


@pytest.mark.gpu
def test_tensors_given_twice():
    x = torch.ones(9, device=DEV)
    assert abs(float(tt.GradientClip(1.0).norm([x, x])[0]) - math.sqrt(18)) <= 5 * U32
    for other in (x, x[3:], x[:1]):
        with pytest.raises(tt.TTEmbError):
            tt.GradientClip(1.0).clip([x, other])
    assert (x == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", [F32, BF16, F16])
def test_adamw_takes_the_factor(kind, bits):
    # a factor that is a power of two: the step of gradients that are that much smaller, bit for bit
    sizes, g = [1000, 3, 70000], ops.gen(5)
    start = [torch.randn(n, device=DEV, generator=g) for n in sizes]
    grads = grads_of(sizes, [kind] * 3, 6)
    for factor in (1.0, 0.25):
        a, b = ([x.clone() for x in start] for _ in range(2))
        one = tt.AdamW(a, lr=1e-2, state_bits=bits, seed=3)
        two = tt.AdamW(b, lr=1e-2, state_bits=bits, seed=3)
        scale = torch.tensor([factor], device=DEV)
        for _ in range(3):
            one.step(grads, grad_scale=scale)
            two.step([x.float() * factor for x in grads])
        for p, q in zip(a + [one.exp_avg.float(), one.exp_avg_sq.float()],
                        b + [two.exp_avg.float(), two.exp_avg_sq.float()]):
            assert torch.equal(p, q)
    p = tt.AdamW([start[0].clone()])
    for bad in (0.5, torch.ones(2, device=DEV), torch.ones(1), torch.ones(1, device=DEV).double()):
        with pytest.raises(tt.TTEmbError):
            p.step([grads[0]], grad_scale=bad)
    assert p.steps == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[50, 3], [300000, 70000]], ids=["one", "many"])
def test_captured_and_on_another_stream(sizes):
    c = tt.GradientClip(1.0)
    grads = grads_of(sizes, [F32, BF16], 9)
    keep = [x.clone() for x in grads]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n0 = c.clip(grads, stream=s)
    s.synchronize()
    ref = [x.clone() for x in grads]
    for x, y in zip(grads, keep):
        x.copy_(y)
    n1 = c.clip(grads)
    assert torch.equal(n0, n1) and all(torch.equal(x, y) for x, y in zip(grads, ref))
    with torch.cuda.stream(s):
        c.clip(grads)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = c.clip(grads)
    for k in range(3):
        for x, y in zip(grads, keep):
            x.copy_(y * (k + 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in grads]
        for x, y in zip(grads, keep):
            x.copy_(y * (k + 1))
        n = c.clip(grads)
        assert torch.equal(n, got) and all(torch.equal(x, y) for x, y in zip(grads, replayed))
