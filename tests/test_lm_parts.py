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


def workspace(n, V, D, dtype):
    best, least = C.c_size_t(), C.c_size_t()
    assert tt.lib().tt_emb_xent_workspace_size(n, V, D, dtype, 1, C.byref(best), C.byref(least)) == 0
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


@pytest.mark.parametrize("dtype", [0, 1])
def test_every_part_begins_in_the_vocabulary(dtype):
    for n, V, D, share in sizes():
        best, least = workspace(n, V, D, dtype)
        parts, _ = tt.tt_emb_xent_parts(n, V, D, dtype, least + int(share * (best - least)))
        assert parts and all(0 <= begin < end <= V for begin, end, _, _ in parts), (n, V, D, share)


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
        assert fn(10, 1000, 200, 1, best, *bad) == tt.TT_EMB_ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("n,V,D", BEHIND)
def test_gradients_where_a_part_ends_with_the_vocabulary(n, V, D, t):
    ops.test_xent_and_gradients(n, V, D, 0, t)
