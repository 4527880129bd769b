"""One operator used by several host threads."""

import threading
import time

import pytest
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt
from tensor_train_compressed_gather_amd import lm


def in_threads(work, count):
    failed = []

    def go(k):
        try:
            work(k)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=go, args=(k,)) for k in range(count)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_calls_of_two_threads_are_enqueued_one_after_the_other(monkeypatch):
    # an entry point that enqueues several kernels, for which it gives up the
    # interpreter, on buffers that grow in between
    op = lm._Operator("cpu")
    monkeypatch.setattr(lm, "_capturing", lambda: False, raising=False)
    inside = []

    def entry(k, ws, size, stream):
        inside.append(k)
        time.sleep(0.002)
        assert inside == [k] and size >= 256 * (k + 1)
        inside.remove(k)
        return 0

    def work(k):
        for i in range(10):
            op._run(entry, "entry", torch.device("cpu"), 1, 256 * (k + 1) * (i + 1), k)

    in_threads(work, 4)


def test_a_refused_call_leaves_the_operator_usable(monkeypatch):
    op = lm._Operator("cpu")
    monkeypatch.setattr(lm, "_capturing", lambda: False, raising=False)
    with pytest.raises(tt.TTEmbError):
        op._run(lambda *a: tt.TT_EMB_ERR_ARG, "entry", torch.device("cpu"), 1, 256)
    op._run(lambda *a: 0, "entry", torch.device("cpu"), 1, 512)


@pytest.mark.gpu
def test_two_threads_on_one_stream_get_their_own_results():
    V, D = 3000, 200
    x, e = tt.VocabCrossEntropy(V, D), tt.TokenEmbedding(V, D)
    cases, refs = [], []
    for k, n in enumerate((50, 700, 333)):
        h, w, target, grad = ops.xent_inputs(n, V, D, torch.bfloat16, 0, n)
        cases.append((h, w, target, grad))
        loss, lse, dh, dw = x.loss_and_grad(h, w, target, grad)
        refs.append((loss, lse, dh, dw.clone(), e.backward(dh, target, grad_weight=dw, accumulate=True)))
    torch.cuda.synchronize()

    def work(k):
        h, w, target, grad = cases[k]
        for _ in range(20):
            got = x.loss_and_grad(h, w, target, grad)
            keep = got[3].clone()
            more = e.backward(got[2], target, grad_weight=got[3], accumulate=True)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip((*got[:3], keep, more), refs[k]))

    in_threads(work, 3)
    assert x.poll_error() == 0 and e.poll_error() == 0
