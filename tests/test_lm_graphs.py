"""Workspaces of the operators around the table under captured graphs: what a
graph writes to stays its own."""

import pytest
import test_lm_ops as ops
import torch

import tensor_train_compressed_gather_amd as tt
from tensor_train_compressed_gather_amd import lm

DEV = ops.DEV


class Buffers(lm._Operator):
    """An operator whose buffers are host memory and whose capture is a flag."""

    def __init__(self, monkeypatch):
        super().__init__("cpu")
        self.capturing = False
        monkeypatch.setattr(lm, "_capturing", lambda: self.capturing, raising=False)

    def __call__(self, need, handle=1):
        return self._workspace(torch.device("cpu"), handle, need)


def test_a_buffer_in_a_graph_is_kept_when_another_replaces_it(monkeypatch):
    op = Buffers(monkeypatch)
    first = op(512)
    assert op(400) is first and not op._kept
    op.capturing = True
    assert op(512) is first
    op.capturing = False
    second = op(4096)  # a larger call on the stream of the capture
    assert second is not first and [b for _, b in op._kept] == [first] and op._kept[0][1] is first
    third = op(8192)   # the second was in no graph: it goes, its status stays readable
    second[:4] = 1
    assert len(op._kept) == 1 and third[:256].sum() == 0
    third[0] = 5
    fourth = op(10000)
    assert fourth[0] == 5 and op(100, handle=2) is not fourth


def test_a_buffer_replaced_inside_a_capture_is_kept(monkeypatch):
    op = Buffers(monkeypatch)
    first = op(512)
    first[0] = 3  # an error that nobody has read
    op.capturing = True
    second = op(4096)
    # no recorded copy from the first, which no replay may read
    assert op._kept[0][1] is first and first[0] == 3 and second[0] == 0
    op.capturing = False
    op(8192)
    assert [b.numel() for _, b in op._kept] == [512, 4096]


@pytest.mark.gpu
def test_a_graph_survives_larger_calls_on_its_stream():
    g = ops.gen(1)
    V, D = 5000, 64
    xe = tt.VocabCrossEntropy(V, D)
    e = tt.TokenEmbedding(V, D)

    def inputs(n):
        return (ops.rows(g, n, D, torch.float32), torch.randint(0, V, (n,), device=DEV, generator=g),
                torch.rand(n, device=DEV, generator=g))

    w = ops.rows(g, V, D, torch.float32)

    def step(h, tok, grad):
        loss, _, dh, dw = xe.loss_and_grad(h, w, tok, grad)
        e.backward(dh, tok, grad_weight=dw, accumulate=True)
        return loss, dh, dw

    small, large = inputs(70), inputs(3000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ref = [x.clone() for x in step(*small)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step(*small)
    for _ in range(3):
        with torch.cuda.stream(s):
            step(*large)  # the workspaces grow
        torch.cuda.synchronize()
        # whatever the allocator gives out now is not what the graph writes to
        other = [torch.full((1 << k,), 7, dtype=torch.uint8, device=DEV) for k in range(12, 26) for _ in range(4)]
        for x in got:
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
        assert all((x == 7).all() for x in other)
    assert xe.poll_error() == 0 and e.poll_error() == 0
    # an error of a replay is in the buffer that the graph kept
    small[1][3] = V
    torch.cuda.synchronize()
    graph.replay()
    assert xe.poll_error() == tt.TT_EMB_ERR_INDEX and xe.poll_error() == 0
    assert e.poll_error() == tt.TT_EMB_ERR_INDEX and e.poll_error() == 0
