"""Token arrays of any shape: the lookup's gradient takes what its forward
gives."""

import pytest
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt


def refused(fn, *args, msg):
    with pytest.raises(tt.TTEmbError) as e:
        fn(*args)
    assert e.value.status == tt.TT_EMB_ERR_ARG and msg in str(e.value), str(e.value)


def test_gradients_of_other_shapes_are_refused():
    e = tt.TokenEmbedding(10, 8)
    tok = torch.zeros((2, 3), dtype=torch.int64)
    # rows at two distances: the library's own error
    refused(e.backward, torch.zeros(3, 2, 8).transpose(0, 1), tok, msg="strides")
    refused(e.backward, torch.zeros(2, 4, 8)[:, :3], tok, msg="strides")
    refused(e.backward, torch.zeros(3, 2, 8), tok, msg="shape")
    refused(e.backward, torch.zeros(8), tok[0], msg="shape")
    refused(e.backward, torch.zeros(()), tok[0], msg="shape")
    refused(e.backward, torch.zeros(9), tok[0, 0], msg="shape")
    # what the kernels could take goes on to the check of the device
    refused(e.backward, torch.zeros(8), tok[0, 0], msg="GPU")
    refused(e.backward, torch.zeros(2, 3, 16)[..., :8], tok, msg="GPU")
    refused(e.backward, torch.zeros(0, 3, 8), tok[:0], msg="GPU")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(), (1,), (4, 5), (2, 3, 4), (0, 3)])
def test_gradient_of_what_forward_gives(shape):
    V, D = 11, 24
    e = tt.TokenEmbedding(V, D, scale=0.5)
    g = ops.gen(3)
    w = ops.rows(g, V, D, torch.float32)
    tok = torch.randint(0, V, shape, device=ops.DEV, generator=g)
    out = e.forward(w, tok)
    assert out.shape == (*shape, D) and torch.equal(out, w[tok] * 0.5)
    wide = torch.zeros((*shape, 2 * D), device=ops.DEV)[..., :D]
    wide.copy_(out)
    for grad in (out, out.reshape(-1, D), wide):
        dw = e.backward(grad, tok)
        flat = e.backward(out.reshape(-1, D), tok.reshape(-1))
        assert torch.equal(dw, flat)
