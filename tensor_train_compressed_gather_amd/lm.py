"""Operators around the table, from token ids to the update of the weights:
embedding lookup with its gradient, layer norm, softmax cross entropy over a
large vocabulary and AdamW (C ABI in ``include/tt_emb.h``).

The classes marshal arguments only: they check what the library cannot see
from raw pointers, allocate outputs on the stream the work runs on, and keep
one workspace per stream.  Matrices may be views whose rows are further apart
than their columns; the last axis has to be contiguous.
"""

from __future__ import annotations

import ctypes as C
import threading

TT_EMB_DTYPE_FLOAT, TT_EMB_DTYPE_BFLOAT, TT_EMB_DTYPE_HALF = 0, 1, 2
TT_EMB_STATUS_BYTES = 256
TT_EMB_XENT_GRAD, TT_EMB_XENT_ALIGNED = 1, 2

LM_EXPORTED = (
    "tt_emb_poll_status",
    "tt_emb_lookup_forward", "tt_emb_lookup_backward", "tt_emb_lookup_workspace_size",
    "tt_emb_norm_forward", "tt_emb_norm_backward", "tt_emb_norm_workspace_size",
    "tt_emb_xent_forward", "tt_emb_xent_loss_grad", "tt_emb_xent_workspace_size", "tt_emb_xent_parts",
    "tt_emb_adamw_update", "tt_emb_adamw_state_size",
)


def declare(L):
    """Argument types of this module's entry points on the loaded library."""
    p, i32, i64, f32, f64, u64, size = (C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_double, C.c_uint64,
                                        C.c_size_t)
    sizes = C.POINTER(size)
    L.tt_emb_poll_status.argtypes = [p, p]
    L.tt_emb_lookup_forward.argtypes = [p, i64, p, i64, i64, i64, i32, f32, p, i64, p, size, p]
    L.tt_emb_lookup_backward.argtypes = [p, i64, p, i64, i64, i64, i32, f32, i64, i32, p, i64, p, size, p]
    L.tt_emb_lookup_workspace_size.argtypes = [i64, i64, i64, sizes]
    L.tt_emb_norm_forward.argtypes = [p, i64, i64, i64, i32, p, p, i32, f32, p, i64, p, p, p]
    L.tt_emb_norm_backward.argtypes = [p, i64, p, i64, i64, i64, i32, p, i32, p, p, p, i64, p, p, p, size, p]
    L.tt_emb_norm_workspace_size.argtypes = [i64, i64, sizes]
    L.tt_emb_xent_forward.argtypes = [p, i64, p, i64, p, i64, i64, i64, i32, i64, p, p, p, size, p]
    L.tt_emb_xent_loss_grad.argtypes = [p, i64, p, i64, p, p, i64, i64, i64, i32, i64, p, p, p, i64, p, i64, p, size,
                                        p]
    L.tt_emb_xent_workspace_size.argtypes = [i64, i64, i64, i32, i32, sizes, sizes]
    L.tt_emb_xent_parts.argtypes = [i64, i64, i64, i32, i32, size, p, i64, C.POINTER(i64), C.POINTER(i32)]
    L.tt_emb_adamw_update.argtypes = [i32, p, p, i32, p, p, p, p, p, p, i32, f64, f64, f64, f64, f64, i64, u64, p]
    L.tt_emb_adamw_state_size.argtypes = [i32, p, C.POINTER(i64)]


torch = None       # imported with the first operator: the package itself does without
_L = _check = None  # the loaded library, the status check
_raw_stream = _capturing = None
_DTYPES = {}


def _bind():
    """Import torch, load the library (once)."""
    global torch, _L, _check, _raw_stream, _capturing
    if _L is None:
        import torch as t

        from . import _check as check, lib

        torch, _check = t, check
        _DTYPES.update({t.float32: 0, t.bfloat16: 1, t.float16: 2})
        # the current stream's handle without a Stream object around it
        _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: t.cuda.current_stream(index).cuda_stream)
        # whether the current stream is being captured into a graph
        _capturing = getattr(t._C, "_cuda_isCurrentStreamCapturing", None) or t.cuda.is_current_stream_capturing
        _L = lib()


def _bad(where: str, what: str, status: int = -1):
    from . import TTEmbError

    return TTEmbError(status, f"{where}: {what}")


def _dtype(t, where: str, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise _bad(where, f"{name}: dtype {t.dtype}, expected float32, bfloat16 or float16")
    return code


def _matrix(t, where: str, name: str, cols: int, rows: int | None = None, dtype=None, device=None):
    """Check a [rows][cols] argument and return the distance of its rows."""
    if not isinstance(t, torch.Tensor):
        raise _bad(where, f"{name}: expected a torch tensor, got {type(t).__name__}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise _bad(where, f"{name}: shape {tuple(shape)}, expected [{'n' if rows is None else rows}, {cols}]")
    if dtype is not None and t.dtype is not dtype:
        raise _bad(where, f"{name}: dtype {t.dtype}, expected {dtype}")
    strides = t.stride()
    ld = strides[0] if shape[0] > 1 else cols
    if (cols > 1 and strides[1] != 1) or ld < cols:
        raise _bad(where, f"{name}: strides {strides}, expected contiguous rows that do not overlap")
    if not t.is_cuda or (device is not None and t.device != device):
        _on(t, where, name, device)
    return ld


def _vector(t, where: str, name: str, length: int, dtypes, device=None):
    if not isinstance(t, torch.Tensor):
        raise _bad(where, f"{name}: expected a torch tensor, got {type(t).__name__}")
    shape = t.shape
    if len(shape) != 1 or shape[0] != length:
        raise _bad(where, f"{name}: shape {tuple(shape)}, expected [{length}]")
    if t.dtype not in dtypes:
        raise _bad(where, f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if length > 1 and t.stride(0) != 1:
        raise _bad(where, f"{name}: not contiguous")
    if not t.is_cuda or (device is not None and t.device != device):
        _on(t, where, name, device)


def _on(t, where: str, name: str, device):
    if t.device.type != "cuda":
        raise _bad(where, f"{name}: on {t.device}, expected a GPU tensor")
    if device is not None and t.device != device:
        raise _bad(where, f"{name}: on {t.device}, expected {device} like the others")


def _guard(device, stream, where: str):
    """What has to be entered before a call's work is enqueued: nothing where
    it goes to the current stream of the current device, else the given
    stream (a torch stream or a handle) or the tensors' device.  Outputs and
    workspaces then belong to the stream that writes them."""
    if stream is None:
        return None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    elif stream.device != device:
        raise _bad(where, f"stream: of {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


class _Operator:
    """What the operators with a workspace share: one growing buffer per
    (device, stream), whose status words are zero from the start.

    A buffer that a captured graph writes to is kept for as long as the
    operator, also when a later call needs a larger one: keep the operator as
    long as the graph.  Make one ordinary call on the stream before the
    capture; a buffer that is first made inside a capture has its status
    cleared by each replay.  Graphs and calls of one stream share its buffer, so
    they may not run at the same time; give graphs that do an operator each.

    Threads may share an operator: a call's kernels are enqueued together, so
    that calls of one stream do not meet in its buffer."""

    def __init__(self, device):
        _bind()
        self.device = torch.device(device)
        self._lock = threading.Lock()
        self._ws = {}
        self._in_graph = set()  # keys whose present buffer a graph writes to
        self._kept = []         # (key, buffer) that graphs write to and no other call any more

    def _workspace(self, device, handle: int, need: int):
        key = (device.index, handle)
        ws = self._ws.get(key)
        capturing = _capturing()
        if ws is None or ws.numel() < need:
            new = torch.empty(need, dtype=torch.uint8, device=device)
            if ws is not None and (capturing or key in self._in_graph):
                # recorded copies and kernels would meet freed memory
                self._kept.append((key, ws))
                self._in_graph.discard(key)
                ws = None
            # the status of earlier calls stays readable
            if ws is None:
                new[:TT_EMB_STATUS_BYTES].zero_()
            else:
                new[:TT_EMB_STATUS_BYTES].copy_(ws[:TT_EMB_STATUS_BYTES])
            self._ws[key] = ws = new
        if capturing:
            self._in_graph.add(key)
        return ws

    def _run(self, fn, where: str, device, handle: int, need: int, *args):
        """Enqueue a call that takes (ws, ws_bytes, stream) behind args."""
        with self._lock:
            ws = self._workspace(device, handle, need)
            rc = fn(*args, ws.data_ptr(), ws.numel(), handle)
        _check(rc, where)

    def poll_error(self) -> int:
        """Synchronises; the first device-detected error of any stream's
        calls since the last poll (0 = ok), cleared by reading it."""
        rc = 0
        with self._lock:
            buffers = [(key, ws, True) for key, ws in self._kept]
            buffers += [(key, ws, key in self._in_graph) for key, ws in self._ws.items()]
        for (index, handle), ws, in_graph in buffers:
            with torch.cuda.device(index):
                if in_graph:
                    torch.cuda.synchronize()  # a graph is replayed on any stream
                got = int(_L.tt_emb_poll_status(ws.data_ptr(), handle))
            rc = rc or got
        return rc


def _size(fn, where: str, *args) -> int:
    out = C.c_size_t()
    _check(fn(*args, C.byref(out)), where)
    return int(out.value)


class TokenEmbedding(_Operator):
    """Rows of a dense [V][D] table for token ids, times ``scale``.

    forward(weight, tokens) -> [*tokens.shape, D] of the weight's type.
    backward(grad_out, tokens), grad_out [n, D] or [*tokens.shape, D] -> the gradient of the weight, summed by sorted
    tokens (bit-reproducible); tokens equal to ``padding_idx`` (negative: none)
    give none.  With accumulate=True it is added to ``grad_weight``, for a
    table that the output layer shares."""

    def __init__(self, V: int, D: int, scale: float = 1.0, padding_idx: int = -1, device="cuda"):
        super().__init__(device)
        self.V, self.D, self.scale, self.padding_idx = int(V), int(D), float(scale), int(padding_idx)
        _size(_L.tt_emb_lookup_workspace_size, "TokenEmbedding", 0, self.V, self.D)

    def _tokens(self, tokens, where, device):
        if not isinstance(tokens, torch.Tensor) or tokens.dtype is not torch.int64:
            raise _bad(where, "tokens: expected an int64 tensor")
        if not tokens.is_contiguous():
            raise _bad(where, "tokens: not contiguous")
        if tokens.device != device:
            _on(tokens, where, "tokens", device)
        return tokens.numel()

    def forward(self, weight, tokens, out=None, stream=None):
        where = "TokenEmbedding.forward"
        ld_w = _matrix(weight, where, "weight", self.D, self.V)
        dt = _dtype(weight, where, "weight")
        device = weight.device
        n = self._tokens(tokens, where, device)
        guard = _guard(device, stream, where)
        if guard is not None:
            with guard:
                return self.forward(weight, tokens, out)
        s = _raw_stream(device.index)
        made = out is None
        if made:
            out, ld_o = weight.new_empty((n, self.D)), self.D
        else:
            ld_o = _matrix(out, where, "out", self.D, n, weight.dtype, device)
        self._run(_L.tt_emb_lookup_forward, where, device, s, TT_EMB_STATUS_BYTES, weight.data_ptr(), ld_w,
                  tokens.data_ptr(), n, self.V, self.D, dt, self.scale, out.data_ptr(), ld_o)
        return out.view(*tokens.shape, self.D) if made and tokens.dim() != 1 else out

    def backward(self, grad_out, tokens, grad_weight=None, accumulate: bool = False, stream=None):
        where = "TokenEmbedding.backward"
        if isinstance(grad_out, torch.Tensor) and grad_out.dim() != 2 and grad_out.dim() > 0:
            if grad_out.shape[:-1] != getattr(tokens, "shape", None):
                raise _bad(where, f"grad_out: shape {tuple(grad_out.shape)}, not that of tokens and {self.D}")
            try:
                grad_out = grad_out.view(tokens.numel(), grad_out.shape[-1])
            except RuntimeError:
                raise _bad(where, f"grad_out: strides {grad_out.stride()}, expected rows at one distance") from None
        ld_g = _matrix(grad_out, where, "grad_out", self.D)
        dt = _dtype(grad_out, where, "grad_out")
        device = grad_out.device
        n = self._tokens(tokens, where, device)
        if grad_out.shape[0] != n:
            raise _bad(where, f"grad_out: {grad_out.shape[0]} rows for {n} tokens")
        if grad_weight is None and accumulate:
            raise _bad(where, "accumulate needs grad_weight")
        need = _size(_L.tt_emb_lookup_workspace_size, where, n, self.V, self.D)
        guard = _guard(device, stream, where)
        if guard is not None:
            with guard:
                return self.backward(grad_out, tokens, grad_weight, accumulate)
        s = _raw_stream(device.index)
        if grad_weight is None:
            grad_weight = torch.empty((self.V, self.D), dtype=grad_out.dtype, device=device)
        ld_w = _matrix(grad_weight, where, "grad_weight", self.D, self.V, grad_out.dtype, device)
        self._run(_L.tt_emb_lookup_backward, where, device, s, need, grad_out.data_ptr(), ld_g, tokens.data_ptr(), n,
                  self.V, self.D, dt, self.scale, self.padding_idx, 1 if accumulate else 0, grad_weight.data_ptr(),
                  ld_w)
        return grad_weight


class LayerNorm(_Operator):
    """Layer norm over rows of D elements.

    forward(x, gamma, beta) -> (y, mean, rstd), y of x's type and the
    statistics fp32; gamma and beta (x's type or fp32) may be None.
    backward(grad_y, x, gamma, mean, rstd) -> (grad_x, dgamma, dbeta), the
    last two of gamma's type (fp32 without gamma)."""

    def __init__(self, D: int, eps: float = 1e-5, device="cuda"):
        super().__init__(device)
        self.D, self.eps = int(D), float(eps)
        _size(_L.tt_emb_norm_workspace_size, "LayerNorm", 0, self.D)

    def _param(self, p, name, where, x):
        if p is not None:
            _vector(p, where, name, self.D, (torch.float32, x.dtype), x.device)

    def forward(self, x, gamma=None, beta=None, out=None, stream=None):
        where = "LayerNorm.forward"
        ld_x = _matrix(x, where, "x", self.D)
        dt = _dtype(x, where, "x")
        n, device = x.shape[0], x.device
        self._param(gamma, "gamma", where, x)
        self._param(beta, "beta", where, x)
        if gamma is not None and beta is not None and gamma.dtype != beta.dtype:
            raise _bad(where, f"beta: dtype {beta.dtype}, expected {gamma.dtype} like gamma")
        param = gamma if gamma is not None else beta
        pdt = 0 if param is None else _dtype(param, where, "gamma")
        guard = _guard(device, stream, where)
        if guard is not None:
            with guard:
                return self.forward(x, gamma, beta, out)
        s = _raw_stream(device.index)
        if out is None:
            out, ld_y = x.new_empty((n, self.D)), self.D
        else:
            ld_y = _matrix(out, where, "out", self.D, n, x.dtype, device)
        mean = torch.empty(n, dtype=torch.float32, device=device)
        rstd = torch.empty(n, dtype=torch.float32, device=device)
        _check(_L.tt_emb_norm_forward(x.data_ptr(), ld_x, n, self.D, dt,
                                    None if gamma is None else gamma.data_ptr(),
                                    None if beta is None else beta.data_ptr(), pdt, self.eps, out.data_ptr(),
                                    ld_y, mean.data_ptr(), rstd.data_ptr(), s), where)
        return out, mean, rstd

    def backward(self, grad_y, x, gamma, mean, rstd, stream=None):
        where = "LayerNorm.backward"
        ld_x = _matrix(x, where, "x", self.D)
        dt = _dtype(x, where, "x")
        n, device = x.shape[0], x.device
        ld_g = _matrix(grad_y, where, "grad_y", self.D, n, x.dtype, device)
        self._param(gamma, "gamma", where, x)
        pdt = 0 if gamma is None else _dtype(gamma, where, "gamma")
        _vector(mean, where, "mean", n, (torch.float32,), device)
        _vector(rstd, where, "rstd", n, (torch.float32,), device)
        need = _size(_L.tt_emb_norm_workspace_size, where, n, self.D)
        guard = _guard(device, stream, where)
        if guard is not None:
            with guard:
                return self.backward(grad_y, x, gamma, mean, rstd)
        s = _raw_stream(device.index)
        dx = x.new_empty((n, self.D))
        kind = torch.float32 if gamma is None else gamma.dtype
        dgamma = torch.empty(self.D, dtype=kind, device=device)
        dbeta = torch.empty(self.D, dtype=kind, device=device)
        self._run(_L.tt_emb_norm_backward, where, device, s, need, grad_y.data_ptr(), ld_g, x.data_ptr(), ld_x, n,
                  self.D, dt, None if gamma is None else gamma.data_ptr(), pdt, mean.data_ptr(), rstd.data_ptr(),
                  dx.data_ptr(), self.D, dgamma.data_ptr(), dbeta.data_ptr())
        return dx, dgamma, dbeta


class tt_emb_xent_part(C.Structure):
    _fields_ = [("begin", C.c_int64), ("end", C.c_int64), ("slot", C.c_int32), ("first", C.c_int32)]


def tt_emb_xent_parts(n: int, V: int, D: int, dtype: int, ws_bytes: int, aligned: bool = False):
    """The parts (begin, end, slot, first) of the vocabulary that
    loss_and_grad sums the hidden rows' gradient over, in order, and how many
    slots it adds up in the end (host-side; the launches use the same
    functions)."""
    _bind()
    count, slots = C.c_int64(), C.c_int32()
    what = TT_EMB_XENT_GRAD | (TT_EMB_XENT_ALIGNED if aligned else 0)
    args = (int(n), int(V), int(D), int(dtype), what, int(ws_bytes))
    _check(_L.tt_emb_xent_parts(*args, None, 0, C.byref(count), C.byref(slots)), "tt_emb_xent_parts")
    parts = (tt_emb_xent_part * count.value)()
    _check(_L.tt_emb_xent_parts(*args, parts, count.value, C.byref(count), C.byref(slots)), "tt_emb_xent_parts")
    return [(q.begin, q.end, q.slot, q.first) for q in parts], int(slots.value)


class VocabCrossEntropy(_Operator):
    """Softmax cross entropy of hidden rows [n][D] against a vocabulary
    [V][D] (both fp32 or both bf16) without keeping the logits.

    forward(hidden, weight, targets) -> (loss, lse), fp32 [n]; 0 where the
    target is ``ignore_index``.
    loss_and_grad(hidden, weight, targets, grad_loss) -> (loss, lse,
    grad_hidden, grad_weight) for fp32 grad_loss [n] = dL/dloss.
    ``max_workspace`` bounds the scratch of loss_and_grad in bytes (smaller
    pieces of the vocabulary at a time).

    fp32 inputs are taken as two fp16 terms, 22 bits: the weight's values with
    one scale for all of them, so beside one of 2^k a value of 1 keeps no more
    than 39 - k bits.  bf16 rows of a multiple of 64 columns that begin at
    multiples of 16 bytes are read in place; other weights are copied by each
    call."""

    def __init__(self, V: int, D: int, ignore_index: int = -100, device="cuda", max_workspace: int | None = None):
        super().__init__(device)
        self.V, self.D, self.ignore_index = int(V), int(D), int(ignore_index)
        self.max_workspace = None if max_workspace is None else int(max_workspace)
        self._need(0, 0, False, "VocabCrossEntropy")

    def _need(self, n: int, dt: int, grad: bool, where: str, aligned: bool = False) -> int:
        best, least = C.c_size_t(), C.c_size_t()
        what = (TT_EMB_XENT_GRAD if grad else 0) | (TT_EMB_XENT_ALIGNED if aligned else 0)
        _check(_L.tt_emb_xent_workspace_size(n, self.V, self.D, dt, what, C.byref(best), C.byref(least)), where)
        if self.max_workspace is None or not grad:
            return int(best.value)
        if self.max_workspace < least.value:
            raise _bad(where, f"max_workspace {self.max_workspace}, at least {least.value} needed", -3)
        return min(int(best.value), self.max_workspace)

    def _inputs(self, hidden, weight, targets, where):
        ld_h = _matrix(hidden, where, "hidden", self.D)
        dt = _dtype(hidden, where, "hidden")
        n, device = hidden.shape[0], hidden.device
        ld_w = _matrix(weight, where, "weight", self.D, self.V, hidden.dtype, device)
        _vector(targets, where, "targets", n, (torch.int64,), device)
        # bf16 operands that lie like this are read in place and need no room for copies
        aligned = (dt == 1 and not (ld_h | ld_w) & 7 and ld_h <= 1 << 20 and ld_w <= 1 << 20
                   and not (hidden.data_ptr() | weight.data_ptr()) & 15)
        return ld_h, ld_w, dt, n, device, aligned

    def forward(self, hidden, weight, targets, stream=None):
        where = "VocabCrossEntropy.forward"
        ld_h, ld_w, dt, n, device, aligned = self._inputs(hidden, weight, targets, where)
        need = self._need(n, dt, False, where, aligned)
        guard = _guard(device, stream, where)
        if guard is not None:
            with guard:
                return self.forward(hidden, weight, targets)
        s = _raw_stream(device.index)
        loss = torch.empty(n, dtype=torch.float32, device=device)
        lse = torch.empty(n, dtype=torch.float32, device=device)
        self._run(_L.tt_emb_xent_forward, where, device, s, need, hidden.data_ptr(), ld_h, weight.data_ptr(), ld_w,
                  targets.data_ptr(), n, self.V, self.D, dt, self.ignore_index, loss.data_ptr(), lse.data_ptr())
        return loss, lse

    def loss_and_grad(self, hidden, weight, targets, grad_loss, grad_weight=None, stream=None):
        where = "VocabCrossEntropy.loss_and_grad"
        ld_h, ld_w, dt, n, device, aligned = self._inputs(hidden, weight, targets, where)
        _vector(grad_loss, where, "grad_loss", n, (torch.float32,), device)
        need = self._need(n, dt, True, where, aligned)
        guard = _guard(device, stream, where)
        if guard is not None:
            with guard:
                return self.loss_and_grad(hidden, weight, targets, grad_loss, grad_weight)
        s = _raw_stream(device.index)
        loss = torch.empty(n, dtype=torch.float32, device=device)
        lse = torch.empty(n, dtype=torch.float32, device=device)
        dh = torch.empty((n, self.D), dtype=hidden.dtype, device=device)
        if grad_weight is None:
            grad_weight = torch.empty((self.V, self.D), dtype=hidden.dtype, device=device)
        ld_dw = _matrix(grad_weight, where, "grad_weight", self.D, self.V, hidden.dtype, device)
        self._run(_L.tt_emb_xent_loss_grad, where, device, s, need, hidden.data_ptr(), ld_h, weight.data_ptr(), ld_w,
                  targets.data_ptr(), grad_loss.data_ptr(), n, self.V, self.D, dt, self.ignore_index, loss.data_ptr(),
                  lse.data_ptr(), dh.data_ptr(), self.D, grad_weight.data_ptr(), ld_dw)
        return loss, lse, dh, grad_weight


class AdamW:
    """AdamW over a list of fp32 tensors, in one launch per 88 of them.

    ``state_bits`` 32 keeps both moments in fp32; 8 keeps them in e4m3 and
    e5m2 with one fp32 scale per 256 elements and rounds at random, from
    ``seed`` and the step's number.  ``copies``: bf16 tensors of the same
    shapes that receive the updated values.  The state is ``exp_avg``,
    ``exp_avg_sq`` (flat; each tensor begins at a multiple of 256 elements),
    ``exp_avg_scale``, ``exp_avg_sq_scale`` and ``steps``.  ``eps`` is at least
    2^-126.  Parameters may be replaced (``param.data = ...``) by tensors of the
    same shape; every step needs a gradient for each."""

    BLOCK = 256

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, copies=None, seed: int = 0):
        _bind()
        where = "AdamW"
        self.params = list(params)
        if not self.params:
            raise _bad(where, "no parameters")
        if state_bits not in (8, 32):
            raise _bad(where, f"state_bits {state_bits}, expected 8 or 32")
        device = None
        for i, p in enumerate(self.params):
            self._tensor(p, f"params[{i}]", torch.float32, None, device)
            device = p.device
        self.copies = None if copies is None else list(copies)
        if self.copies is not None:
            if len(self.copies) != len(self.params):
                raise _bad(where, f"{len(self.copies)} copies for {len(self.params)} parameters")
            for i, (c, p) in enumerate(zip(self.copies, self.params)):
                self._tensor(c, f"copies[{i}]", torch.bfloat16, p.shape, device)
        self.lr, self.betas, self.eps, self.weight_decay = float(lr), tuple(betas), float(eps), float(weight_decay)
        self.state_bits, self.seed, self.steps, self.device = int(state_bits), int(seed), 0, device
        n = len(self.params)
        self._array = C.c_void_p * n
        self._numel = (C.c_int64 * n)(*[p.numel() for p in self.params])
        self._shapes = [p.shape for p in self.params]
        total = C.c_int64()
        _check(_L.tt_emb_adamw_state_size(n, self._numel, C.byref(total)), where)
        length = int(total.value)
        kinds = (torch.float32, torch.float32) if state_bits == 32 else (torch.float8_e4m3fn, torch.float8_e5m2)
        size = 4 if state_bits == 32 else 1
        self.exp_avg, self.exp_avg_sq = (torch.zeros(length * size, dtype=torch.uint8, device=device).view(k)
                                         for k in kinds)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        if state_bits == 8:
            self.exp_avg_scale = torch.zeros(length // self.BLOCK, dtype=torch.float32, device=device)
            self.exp_avg_sq_scale = torch.zeros_like(self.exp_avg_scale)

    @staticmethod
    def _tensor(t, name, dtype, shape, device):
        where = "AdamW"
        if not torch.is_tensor(t):
            raise _bad(where, f"{name}: expected a torch tensor, got {type(t).__name__}")
        if t.dtype != dtype:
            raise _bad(where, f"{name}: dtype {t.dtype}, expected {dtype}")
        if shape is not None and t.shape != shape:
            raise _bad(where, f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise _bad(where, f"{name}: not contiguous")
        _on(t, where, name, device)

    def _whole(self, tensors, name, dtype):
        """Check that the kernel can take these for the parameters' elements."""
        tensor, index = torch.Tensor, self.device.index
        if len(tensors) != len(self._shapes):
            raise _bad("AdamW", f"{len(tensors)} {name} for {len(self._shapes)} parameters")
        for t, shape in zip(tensors, self._shapes):
            if (not isinstance(t, tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
                    or t.get_device() != index):
                break
        else:
            return
        for i, (t, shape) in enumerate(zip(tensors, self._shapes)):
            self._tensor(t, f"{name}[{i}]", dtype, shape, self.device)

    def load_state(self, exp_avg, exp_avg_sq, steps: int, exp_avg_scale=None, exp_avg_sq_scale=None):
        """Copies of a saved state: the moments (and scales) as this class
        keeps them, and the number of steps taken."""
        for mine, given, name in ((self.exp_avg, exp_avg, "exp_avg"), (self.exp_avg_sq, exp_avg_sq, "exp_avg_sq"),
                                  (self.exp_avg_scale, exp_avg_scale, "exp_avg_scale"),
                                  (self.exp_avg_sq_scale, exp_avg_sq_scale, "exp_avg_sq_scale")):
            if (mine is None) != (given is None) or (mine is not None and (mine.shape != given.shape
                                                                           or mine.dtype != given.dtype)):
                raise _bad("AdamW.load_state", f"{name} does not match this state")
        if int(steps) < 0:
            raise _bad("AdamW.load_state", "steps is negative")
        self.exp_avg.copy_(exp_avg)
        self.exp_avg_sq.copy_(exp_avg_sq)
        if self.exp_avg_scale is not None:
            self.exp_avg_scale.copy_(exp_avg_scale)
            self.exp_avg_sq_scale.copy_(exp_avg_sq_scale)
        self.steps = int(steps)

    def step(self, grads, lr: float | None = None, stream=None):
        """One update from gradients shaped like the parameters (all of one
        type: fp32, bf16 or fp16)."""
        where = "AdamW.step"
        grads = list(grads)
        n = len(self._shapes)
        if len(grads) != n:
            raise _bad(where, f"{len(grads)} gradients for {n} parameters")
        first = getattr(grads[0], "dtype", None)
        self._whole(grads, "grads", first)
        dt = _dtype(grads[0], where, "grads[0]")
        # parameters may have been replaced (param.data = ...): they are checked and their addresses read anew
        self._whole(self.params, "params", torch.float32)
        if self.copies is not None:
            self._whole(self.copies, "copies", torch.bfloat16)
        array, address = self._array, torch.Tensor.data_ptr
        params = array(*map(address, self.params))
        pointers = array(*map(address, grads))
        copies = None if self.copies is None else array(*map(address, self.copies))
        guard = _guard(self.device, stream, where)
        if guard is not None:
            with guard:
                return self.step(grads, lr)
        s = _raw_stream(self.device.index)
        _check(_L.tt_emb_adamw_update(
            n, params, pointers, dt, copies, self._numel, self.exp_avg.data_ptr(), self.exp_avg_sq.data_ptr(),
            None if self.exp_avg_scale is None else self.exp_avg_scale.data_ptr(),
            None if self.exp_avg_sq_scale is None else self.exp_avg_sq_scale.data_ptr(), self.state_bits,
            self.lr if lr is None else float(lr), self.betas[0], self.betas[1], self.eps, self.weight_decay,
            self.steps + 1, self.seed & 0xFFFFFFFFFFFFFFFF, s), where)
        self.steps += 1
