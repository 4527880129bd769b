"""Refusals of the operators around the table that need no GPU: the C entry
points check their arguments before any device work, and the binding refuses
what the library would misread."""

import ctypes as C

import pytest
import torch

import tensor_train_compressed_gather_amd as tt
from tensor_train_compressed_gather_amd import lm

ARG, WS, UNSUPPORTED = tt.TT_EMB_ERR_ARG, tt.TT_EMB_ERR_WORKSPACE, tt.TT_EMB_ERR_UNSUPPORTED
P, Q, R = 0x10000, 0x20000, 0x30000  # addresses that are never read: each call is refused
W = 0x100000                          # a 256-byte aligned workspace address
BIG = 1 << 40


def call(name, good, **bad):
    """The status of an entry point for the good arguments with some replaced."""
    args = dict(good)
    for k, v in bad.items():
        assert k in args, k
        args[k] = v
    return getattr(tt.lib(), name)(*args.values())


LOOKUP_F = dict(weight=P, ld_weight=8, tokens=Q, n=4, V=10, D=8, dtype=0, scale=1.0, out=R, ld_out=8, ws=W,
                ws_bytes=256, stream=None)
LOOKUP_B = dict(grad=P, ld_grad=8, tokens=Q, n=4, V=10, D=8, dtype=0, scale=1.0, pad=-1, acc=0, dw=R, ld_dw=8, ws=W,
                ws_bytes=BIG, stream=None)
NORM_F = dict(x=P, ld_x=8, n=4, D=8, dtype=1, gamma=Q, beta=Q, pdt=0, eps=1e-5, y=R, ld_y=8, mean=None, rstd=None,
              stream=None)
NORM_B = dict(dy=P, ld_dy=8, x=P, ld_x=8, n=4, D=8, dtype=1, gamma=Q, pdt=0, mean=Q, rstd=Q, dx=R, ld_dx=8, dg=None,
              db=None, ws=W, ws_bytes=BIG, stream=None)
XENT_F = dict(h=P, ld_h=8, w=Q, ld_w=8, t=R, n=4, V=10, D=8, dtype=1, ignore=-100, loss=P, lse=P, ws=W, ws_bytes=BIG,
              stream=None)
XENT_G = dict(h=P, ld_h=8, w=Q, ld_w=8, t=R, g=R, n=4, V=10, D=8, dtype=1, ignore=-100, loss=P, lse=P, dh=P, ld_dh=8,
              dw=Q, ld_dw=8, ws=W, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("name,good,bad,code", [
    ("tt_emb_lookup_forward", LOOKUP_F, dict(weight=None), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(weight=P + 2), ARG),       # fp32 off its 4 bytes
    ("tt_emb_lookup_forward", LOOKUP_F, dict(tokens=None), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(out=None), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(ld_weight=7), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(ld_out=7), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(n=-1), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(V=0), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(D=0), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(dtype=3), ARG),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(D=65537, ld_weight=65537, ld_out=65537), UNSUPPORTED),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(V=2 ** 31), UNSUPPORTED),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(ws=None), WS),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(ws=W + 64), WS),
    ("tt_emb_lookup_forward", LOOKUP_F, dict(ws_bytes=255), WS),
    ("tt_emb_lookup_backward", LOOKUP_B, dict(grad=None), ARG),
    ("tt_emb_lookup_backward", LOOKUP_B, dict(dw=None), ARG),
    ("tt_emb_lookup_backward", LOOKUP_B, dict(ld_grad=7), ARG),
    ("tt_emb_lookup_backward", LOOKUP_B, dict(ld_dw=7), ARG),
    ("tt_emb_lookup_backward", LOOKUP_B, dict(tokens=None), ARG),
    ("tt_emb_lookup_backward", LOOKUP_B, dict(ws_bytes=256), WS),
    ("tt_emb_norm_forward", NORM_F, dict(x=None), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(x=P + 1), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(y=None), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(ld_x=7), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(ld_y=7), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(pdt=2), ARG),                  # neither x's type nor fp32
    ("tt_emb_norm_forward", NORM_F, dict(gamma=Q + 2), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(eps=-1.0), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(eps=float("nan")), ARG),
    ("tt_emb_norm_forward", NORM_F, dict(D=16385, ld_x=16385, ld_y=16385), UNSUPPORTED),
    ("tt_emb_norm_backward", NORM_B, dict(mean=None), ARG),
    ("tt_emb_norm_backward", NORM_B, dict(rstd=None), ARG),
    ("tt_emb_norm_backward", NORM_B, dict(dx=None), ARG),
    ("tt_emb_norm_backward", NORM_B, dict(ld_dy=7), ARG),
    ("tt_emb_norm_backward", NORM_B, dict(dg=Q + 2), ARG),
    ("tt_emb_norm_backward", NORM_B, dict(ws_bytes=300), WS),
    ("tt_emb_xent_forward", XENT_F, dict(h=None), ARG),
    ("tt_emb_xent_forward", XENT_F, dict(w=None), ARG),
    ("tt_emb_xent_forward", XENT_F, dict(t=None), ARG),
    ("tt_emb_xent_forward", XENT_F, dict(loss=None), ARG),
    ("tt_emb_xent_forward", XENT_F, dict(lse=None), ARG),
    ("tt_emb_xent_forward", XENT_F, dict(ld_w=7), ARG),
    ("tt_emb_xent_forward", XENT_F, dict(dtype=2), UNSUPPORTED),
    ("tt_emb_xent_forward", XENT_F, dict(D=16385, ld_h=16385, ld_w=16385), UNSUPPORTED),
    ("tt_emb_xent_forward", XENT_F, dict(ws_bytes=256), WS),
    ("tt_emb_xent_forward", XENT_F, dict(n=2 ** 20, V=2 ** 20), UNSUPPORTED),  # more tiles than a launch takes
    ("tt_emb_xent_loss_grad", XENT_G, dict(g=None), ARG),
    ("tt_emb_xent_loss_grad", XENT_G, dict(dh=None), ARG),
    ("tt_emb_xent_loss_grad", XENT_G, dict(dw=None), ARG),
    ("tt_emb_xent_loss_grad", XENT_G, dict(ld_dh=7), ARG),
    ("tt_emb_xent_loss_grad", XENT_G, dict(ld_dw=7), ARG),
    ("tt_emb_xent_loss_grad", XENT_G, dict(ws_bytes=4096), WS),
])
def test_entry_points_refuse(name, good, bad, code):
    assert call(name, good, **bad) == code


def adam(**bad):
    one = C.c_void_p * 1
    good = dict(count=1, params=one(P), grads=one(Q), gdt=0, copies=None, numel=(C.c_int64 * 1)(10), m=R, v=R,
                ms=None, vs=None, bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, seed=0, stream=None)
    return call("tt_emb_adamw_update", good, **bad)


def test_adamw_refuses():
    one = C.c_void_p * 1
    for bad in (dict(count=-1), dict(params=None), dict(grads=None), dict(params=one(None)), dict(grads=one(None)),
                dict(params=one(P + 2)), dict(gdt=5), dict(copies=one(None)), dict(copies=one(P + 1)), dict(m=None),
                dict(v=None), dict(m=R + 4), dict(bits=16), dict(bits=8), dict(lr=-1.0), dict(lr=float("nan")),
                dict(b1=1.0), dict(b2=-0.1), dict(eps=0.0), dict(eps=1e-60), dict(wd=-1.0), dict(step=0),
                dict(numel=(C.c_int64 * 1)(-1)), dict(numel=None)):
        assert adam(**bad) == ARG, bad
    assert adam(count=0) == tt.TT_EMB_OK
    assert adam(numel=(C.c_int64 * 1)(0)) == tt.TT_EMB_OK  # nothing to do, nothing read
    assert adam(numel=(C.c_int64 * 1)(2 ** 50)) == UNSUPPORTED


def test_sizes():
    L = tt.lib()
    out, least, n = C.c_size_t(), C.c_size_t(), C.c_int64()
    assert L.tt_emb_lookup_workspace_size(0, 1, 1, C.byref(out)) == 0 and out.value >= 256
    assert L.tt_emb_lookup_workspace_size(10, 10, 10, None) == ARG
    assert L.tt_emb_lookup_workspace_size(10, 0, 10, C.byref(out)) == ARG
    assert L.tt_emb_norm_workspace_size(10, 16385, C.byref(out)) == UNSUPPORTED
    assert L.tt_emb_norm_workspace_size(10, 100, C.byref(out)) == 0 and out.value >= 256 + 2 * 10 * 100 * 4
    assert L.tt_emb_xent_workspace_size(10, 1000, 64, 1, 1, C.byref(out), C.byref(least)) == 0
    assert 256 <= least.value <= out.value
    assert L.tt_emb_xent_workspace_size(10, 1000, 64, 1, 0, C.byref(out), None) == 0
    assert L.tt_emb_xent_workspace_size(10, 1000, 64, 1, 0, None, None) == ARG
    assert L.tt_emb_xent_workspace_size(10, 1000, 64, 2, 0, C.byref(out), None) == UNSUPPORTED
    sizes = (C.c_int64 * 3)(1, 256, 257)
    assert L.tt_emb_adamw_state_size(3, sizes, C.byref(n)) == 0 and n.value == 4 * 256
    assert L.tt_emb_adamw_state_size(3, None, C.byref(n)) == ARG
    assert L.tt_emb_poll_status(None, None) == ARG


def refused(fn, *args, msg, **kw):
    with pytest.raises(tt.TTEmbError) as e:
        fn(*args, **kw)
    assert e.value.status == ARG and msg in str(e.value), str(e.value)


def test_binding_refuses_what_the_kernels_would_misread():
    w, tok = torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64)
    e = tt.TokenEmbedding(10, 8)
    refused(e.forward, w, tok, msg="GPU")
    refused(e.forward, w.double(), tok, msg="GPU")
    refused(e.forward, torch.zeros(10, 9), tok, msg="shape")
    refused(e.forward, torch.zeros(8, 10).t(), tok, msg="strides")
    refused(e.forward, [1.0], tok, msg="torch tensor")
    refused(e.backward, torch.zeros(8), tok, msg="shape")
    ln = tt.LayerNorm(8)
    refused(ln.forward, torch.zeros(4, 8), msg="GPU")
    refused(ln.forward, torch.zeros(4, 7), msg="shape")
    refused(ln.forward, torch.zeros(8), msg="shape")
    xe = tt.VocabCrossEntropy(10, 8)
    refused(xe.forward, torch.zeros(4, 8), w, tok, msg="GPU")
    refused(xe.forward, torch.zeros(4, 9), w, tok, msg="shape")
    refused(tt.AdamW, [], msg="no parameters")
    refused(tt.AdamW, [torch.zeros(4)], msg="GPU")
    refused(tt.AdamW, [torch.zeros(4).double()], msg="dtype")
    refused(tt.AdamW, [torch.zeros(4, 4).t()[1:]], msg="contiguous")
    refused(tt.AdamW, [torch.zeros(4)], state_bits=16, msg="state_bits")
    for bad in ((0, 8), (10, 0)):
        refused(tt.TokenEmbedding, *bad, msg="")
        refused(tt.VocabCrossEntropy, *bad, msg="")
    with pytest.raises(tt.TTEmbError) as err:
        tt.LayerNorm(16385)
    assert err.value.status == UNSUPPORTED


def test_binding_declares_every_entry_point():
    assert set(lm.LM_EXPORTED) <= set(tt.EXPORTED)
    for name in lm.LM_EXPORTED:
        assert getattr(tt.lib(), name).argtypes is not None, name


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("n,V,D", [(0, 1, 1), (1, 1, 1), (0, 2 ** 31 - 2, 16384), (129, 300, 128),
                                   (60, 2 ** 30 - 2, 16384), (100000, 10 ** 6, 129), (2 ** 30, 100, 8)])
def test_xent_workspace_of_any_size(n, V, D, dtype):
    best, least = C.c_size_t(), C.c_size_t()
    for grad in (0, 1):
        assert tt.lib().tt_emb_xent_workspace_size(n, V, D, dtype, grad, C.byref(best), C.byref(least)) == 0
        assert 256 <= least.value <= best.value
