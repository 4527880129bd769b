"""The parts that the vocabulary cross entropy sums the hidden rows' gradient
over: the plan that the launches follow, walked on the CPU, and results at
sizes where parts end at the vocabulary's end or pieces are unequal."""

import ctypes as C
import random

import pytest
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt

F32, BF16 = torch.float32, torch.bfloat16


def workspace(n, V, D, dtype, aligned=False):
    best, least = C.c_size_t(), C.c_size_t()
    what = 3 if aligned else 1
    assert tt.lib().tt_emb_xent_workspace_size(n, V, D, dtype, what, C.byref(best), C.byref(least)) == 0
    return best.value, least.value


# V a little more than a whole number of parts, where rounding to whole tiles
# would begin one more
BEHIND = [(64, 130740, 256), (64, 130740, 200), (64, 6320, 256), (64, 6320, 200)]
# pieces of which a later, shorter one could be cut into more parts than the first
UNEQUAL = [(768, 256000, 256), (768, 151936, 256), (768, 152064, 256), (768, 250002, 256), (1100, 117700, 256)]


def sizes():
    """Sizes over the operator's range, each with several workspaces."""
    rng = random.Random(7)
    got = [(*s, w) for s in BEHIND + UNEQUAL for w in (0.0, 0.2, 0.5, 0.8, 1.0)]
    got += [(64, 20500, 256, w) for w in (0.0, 0.1, 0.3, 0.6, 1.0)]
    for _ in range(1500):
        n, D = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(4, 12.5))
        V = max(1, min(int(2 ** rng.uniform(5, 20)), 2 ** 32 // n))
        got.append((n, V, D, rng.choice([0.0, 0.3, rng.random(), 1.0])))
    return got


@pytest.mark.parametrize("dtype,aligned", [(0, False), (1, False), (1, True)])
def test_every_part_begins_in_the_vocabulary(dtype, aligned):
    for n, V, D, share in sizes():
        best, least = workspace(n, V, D, dtype, aligned)
        parts, _ = tt.tt_emb_xent_parts(n, V, D, dtype, least + int(share * (best - least)), aligned)
        assert parts and all(0 <= begin < end <= V for begin, end, _, _ in parts), (n, V, D, share)


@pytest.mark.parametrize("dtype,aligned", [(0, False), (1, False), (1, True)])
def test_every_row_is_in_one_part_and_every_part_is_summed(dtype, aligned):
    several = 0
    for n, V, D, share in sizes():
        best, least = workspace(n, V, D, dtype, aligned)
        parts, slots = tt.tt_emb_xent_parts(n, V, D, dtype, least + int(share * (best - least)), aligned)
        at, written = 0, set()
        for begin, end, slot, first in parts:
            assert begin == at, (n, V, D, share)
            at = end
            # a slot is overwritten once, before it is added to, and summed in the end
            assert 0 <= slot < slots and bool(first) == (slot not in written), (n, V, D, share, slot)
            written.add(slot)
        assert at == V and len(written) == slots, (n, V, D, share)
        several += len(parts) > slots > 1  # several pieces and splits
    assert several > 50


def test_parts_are_refused_like_the_call():
    best, least = workspace(10, 1000, 200, 1)
    count, slots = C.c_int64(), C.c_int32()
    fn = tt.lib().tt_emb_xent_parts
    for n, V, D, dtype, ws, code in ((10, 1000, 200, 1, least - 1, tt.TT_EMB_ERR_WORKSPACE),
                                     (0, 1000, 200, 1, best, tt.TT_EMB_ERR_ARG), (10, 0, 200, 1, best, tt.TT_EMB_ERR_ARG),
                                     (10, 1000, 200, 2, best, tt.TT_EMB_ERR_UNSUPPORTED)):
        with pytest.raises(tt.TTEmbError) as e:
            tt.tt_emb_xent_parts(n, V, D, dtype, ws)
        assert e.value.status == code
    for bad in ((None, 1, C.byref(count), C.byref(slots)), (None, -1, C.byref(count), C.byref(slots)),
                (None, 0, None, C.byref(slots)), (None, 0, C.byref(count), None)):
        assert fn(10, 1000, 200, 1, 1, best, *bad) == tt.TT_EMB_ERR_ARG
    for what in (0, 2, 4, 5):  # the parts are those of the call with gradients
        assert fn(10, 1000, 200, 1, what, best, None, 0, C.byref(count), C.byref(slots)) == tt.TT_EMB_ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D", BEHIND)
def test_gradients_where_a_part_ends_with_the_vocabulary(n, V, D, t):
    ops.test_xent_and_gradients(n, V, D, 0, t)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D", UNEQUAL)
def test_gradients_of_unequal_pieces(n, V, D, t):
    # the tolerance of a row's gradient is far below its target's share, which
    # is lost with the part that the target lies in
    h, w, target, grad = ops.xent_inputs(n, V, D, t, 0, V)
    target[::2] = V - 1 - target[::2] % 300  # the last rows
    z, lse, loss, d, mag = ops.xent_reference(h, w, target, grad, -100)
    x = tt.VocabCrossEntropy(V, D)
    got = x.loss_and_grad(h, w, target, grad)
    check_gradients(got, h, w, z, lse, d, mag, t)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D", [(64, 20500, 256), (150, 3000, 200), (300, 9001, 264), (64, 20500, 200)])
def test_gradients_in_pieces_with_every_workspace(n, V, D, t):
    h, w, target, grad = ops.xent_inputs(n, V, D, t, 0, n + V)
    z, lse, loss, d, mag = ops.xent_reference(h, w, target, grad, -100)
    best, least = workspace(n, V, D, int(t == BF16))
    for share in (0.0, 0.1, 0.2, 0.3, 0.6, 1.0):
        x = tt.VocabCrossEntropy(V, D, max_workspace=least + int(share * (best - least)))
        got = x.loss_and_grad(h, w, target, grad)
        check_gradients(got, h, w, z, lse, d, mag, t)
        again = x.loss_and_grad(h, w, target, grad)
        assert all(torch.equal(p, q) for p, q in zip(got, again))


def check_gradients(got, h, w, z, lse, d, mag, t):
    """The bounds of ops.test_xent_and_gradients."""
    (n, D), V = h.shape, w.shape[0]
    h64, w64, U32 = h.double(), w.double(), ops.U32
    ez = ((6 * D if t == F32 else D) + 8) * U32 * (h64.abs() @ w64.abs().t()).amax(1)
    ex = U32 * (4 + 2 * (z - lse[:, None]).abs().amax(1))
    es = ez + ex + (200 + V / 1024) * U32
    ed = ((ops.u(BF16) if t == BF16 else 2.0 ** -23) + ez + es + ex)[:, None] * mag
    k = 6 if t == F32 else 1
    ref = d @ w64
    ops.close(got[2], ref, ed @ w64.abs() + k * (V + 8) * U32 * (mag @ w64.abs()) + ops.u(t) * ref.abs(), "dh")
    ref = d.t() @ h64
    ops.close(got[3], ref, ed.t() @ h64.abs() + k * (n + 8) * U32 * (mag.t() @ h64.abs()) + ops.u(t) * ref.abs(), "dw")
