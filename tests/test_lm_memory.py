"""Workspaces of the vocabulary cross entropy: room for copies of the operands
only where they are made."""

import ctypes as C

import pytest
import test_lm_abi as abi
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

F32, BF16 = torch.float32, torch.bfloat16
GRAD, ALIGNED = 1, 2
MB = 1 << 20


def sizes(n, V, D, dtype, what):
    best, least = C.c_size_t(), C.c_size_t()
    assert tt.lib().tt_emb_xent_workspace_size(n, V, D, dtype, what, C.byref(best), C.byref(least)) == 0
    return best.value, least.value


def test_few_rows_take_no_copy_of_the_weight():
    V, D = 131072, 4096
    assert sizes(1, V, D, 0, 0)[0] < 16 * MB and sizes(128, V, D, 0, 0)[0] < 16 * MB
    assert sizes(129, V, D, 0, 0)[0] > V * D * 4
    assert sizes(5, V, D, 1, ALIGNED)[0] < 16 * MB and sizes(5, V, D, 1, 0)[0] > V * D * 2
    # with gradients: d and the hidden rows' copy
    best = sizes(8192, V, D, 1, GRAD | ALIGNED)[0]
    assert best < 600 * MB and sizes(8192, V, D, 1, GRAD)[0] == best + V * D * 2
    # columns that no tile loads as they are, and fp32 terms
    for D, dtype in ((4095, 1), (200, 1), (4096, 0)):
        assert sizes(300, 1000, D, dtype, ALIGNED) == sizes(300, 1000, D, dtype, 0)
        assert sizes(300, 1000, D, dtype, GRAD | ALIGNED) == sizes(300, 1000, D, dtype, GRAD)


def test_unknown_sizes_are_refused():
    out = C.c_size_t()
    for what in (4, -1, 7):
        assert tt.lib().tt_emb_xent_workspace_size(5, 100, 64, 1, what, C.byref(out), None) == tt.TT_EMB_ERR_ARG


@pytest.mark.parametrize("name,good", [("tt_emb_xent_forward", abi.XENT_F), ("tt_emb_xent_loss_grad", abi.XENT_G)])
def test_operands_that_need_a_copy_are_refused_room_for_none(name, good):
    n, V, D = 600, 4000, 256
    grad = GRAD if "t_emb_xent_loss" in name else 0
    good = dict(good, n=n, V=V, D=D, ld_h=D, ld_w=D, ws_bytes=sizes(n, V, D, 1, grad | ALIGNED)[1])
    if grad:
        good.update(ld_dh=D, ld_dw=D)
    for bad in (dict(w=abi.Q + 2), dict(w=abi.Q + 8), dict(ld_w=D + 4), dict(ld_w=(1 << 20) + 8)):
        assert abi.call(name, good, **bad) == tt.TT_EMB_ERR_WORKSPACE, bad
    if not grad:
        for bad in (dict(h=abi.P + 2), dict(ld_h=D + 1)):
            assert abi.call(name, good, **bad) == tt.TT_EMB_ERR_WORKSPACE, bad


@pytest.mark.gpu
@pytest.mark.parametrize("n", [5, 300])
def test_scores_and_gradients_of_operands_however_they_lie(n):
    V, D = 2500, 256
    h, w, target, grad = ops.xent_inputs(n, V, D, BF16, 0, n)
    x = tt.VocabCrossEntropy(V, D)

    def lie(a, gap, at):
        flat = torch.zeros(a.shape[0] * (D + gap) + at, device=ops.DEV, dtype=a.dtype)
        view = flat[at:].view(a.shape[0], D + gap)[:, :D]
        view.copy_(a)
        return view

    ref = x.forward(h, w, target)
    small = sum(b.numel() for b in x._ws.values())
    assert small < 4 * n * V + 65536  # no copy of the weight
    ref_grad = x.loss_and_grad(h, w, target, grad)
    for gap, at in ((8, 0), (0, 8), (4, 0), (0, 4), (1, 3)):
        for a, b in ((h, lie(w, gap, at)), (lie(h, gap, at), w), (lie(h, gap, at), lie(w, gap, at))):
            y = tt.VocabCrossEntropy(V, D)
            for op in (x, y):
                assert all(torch.equal(p, q) for p, q in zip(op.forward(a, b, target), ref))
                assert all(torch.equal(p, q) for p, q in zip(op.loss_and_grad(a, b, target, grad), ref_grad))
