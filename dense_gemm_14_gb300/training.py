"""Tensor-level calls of the training products: softmax cross entropy over a
projection's outputs, activations kept in 8 bits, rows of a table looked up by
token and their gradient, and the norm of many gradients and their clipping
(argument marshalling only; every step runs in the library's CUDA kernels). None
of them is recorded by autograd."""
from __future__ import annotations

import math

import torch

from . import _lib
from .api import (_CODE, _FP32_MODES, _capturing, _graph_workspace, _workspace, _workspace_lock,
                  _workspaces)

_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice  # (of a context that operands' tensors have made)

CKPT8_BLOCK = 32  # columns of a row that share a scale


def _code(x: torch.Tensor, fp32_mode: str | None) -> int:
    if x.dtype not in _CODE:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if fp32_mode not in _FP32_MODES or (fp32_mode not in (None, "fp32") and x.dtype != torch.float32):
        raise ValueError(f"fp32_mode {fp32_mode!r} needs float32 inputs and one of {list(_FP32_MODES)}")
    return _FP32_MODES[fp32_mode] if x.dtype == torch.float32 else _CODE[x.dtype]


def _on(stream, device: torch.device, body):
    """body(stream handle) with `device` and, where one is given, `stream`
    current: what the call allocates then belongs to the stream its kernels run on."""
    if stream is None:
        # the handle itself: making a Stream object of it takes as long as a launch
        if device.index == _current_device():
            return body(_current_stream(device.index))
        with torch.cuda.device(device):
            return body(_current_stream(device.index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _in_workspace(device: torch.device, handle: int, call, need, where: str) -> None:
    """call(workspace pointer, bytes) on the stream's workspace as it is; where
    it is refused, on one of need() bytes (asked for only then). A call that
    fails otherwise may have run in part, and is not repeated. In a graph being
    captured: on memory of the graph's own."""
    with _workspace_lock(device, handle):
        capturing = _capturing()
        ws = None if capturing else _workspaces.get((device.index, handle))
        if ws is not None:
            status = call(ws.data_ptr(), ws.numel())
            if status == _lib.GEMM14_OK:
                return
            if status != _lib.GEMM14_ERR_INVALID_ARG:
                raise _lib.Gemm14Error(status, where)
        n = need()
        make = _graph_workspace if capturing else _workspace
        ws = make(device, handle, n) if n else None
        status = call(ws.data_ptr() if n else None, ws.numel() if n else 0)
        if status:
            raise _lib.Gemm14Error(status, where)


def _matrix(x: torch.Tensor, name: str, device: int | None = None) -> int:
    """The row pitch of a row-major CUDA matrix (on the device of this index)."""
    if not x.is_cuda or (device is not None and x.get_device() != device):
        raise ValueError(f"{name} must be a CUDA tensor on the operands' device")
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(x.shape)}")
    (rows, cols), (pitch, step) = x.shape, x.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have unit stride along its rows (row-major)")
    if rows <= 1 or cols == 0:
        return max(cols, 1)
    if pitch < cols:
        raise ValueError(f"{name}: rows overlap (stride {x.stride()})")
    return pitch


def _vector(x: torch.Tensor, name: str, n: int, dtype: torch.dtype, device: int) -> None:
    if x.get_device() != device or x.dtype != dtype or x.shape != (n,) or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA vector of {n} values on the "
                         f"operands' device, got {x.dtype} {tuple(x.shape)} on {x.device}")


def _ptr(x: torch.Tensor | None) -> int | None:
    return x.data_ptr() if x is not None and x.numel() else None


def _ce_operands(h, w, targets, fp32_mode):
    code = _code(h, fp32_mode)
    if w.dtype != h.dtype:
        raise TypeError(f"h and w differ in dtype: {h.dtype}, {w.dtype}")
    device = h.get_device()
    ldh, ldw = _matrix(h, "h"), _matrix(w, "w", device)
    (T, D), (V, D2) = h.shape, w.shape
    if D != D2 or V < 1 or D < 1:
        raise ValueError(f"shape mismatch: h {tuple(h.shape)}, w {tuple(w.shape)}")
    _vector(targets, "targets", T, torch.int64, device)
    return code, T, V, D, ldh, ldw


def linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                         ignore_index: int = -100, stream=None, fp32_mode: str | None = None
                         ) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse) of softmax cross entropy on the logits h @ w.T, which are
    formed in pieces of the vocabulary and never kept (gemm14_linear_ce_forward).

    h: (T, D) and w: (V, D) in float32, bfloat16 or float16, row-major views on
    one GPU; targets: (T,) int64. loss, lse: (T,) float32, 0 for rows whose
    target is ignore_index; a target outside [0, V) gives NaN. Keep lse for
    linear_cross_entropy_backward. Runs on `stream` (default: torch's current
    stream) without synchronising, with a workspace cached per (device, stream)
    (in a graph being captured, memory of the graph's own); what it allocates belongs to that stream, and operands made on another are
    the caller's to order and keep (wait_stream, record_stream). Not recorded by
    autograd: linear_cross_entropy_backward forms the gradients.
    fp32_mode as for gemm_into."""
    code, T, V, D, ldh, ldw = _ce_operands(h, w, targets, fp32_mode)

    def body(handle):
        loss = torch.empty(T, dtype=torch.float32, device=h.device)
        lse = torch.empty(T, dtype=torch.float32, device=h.device)
        if T:
            hp, wp = h.data_ptr(), w.data_ptr()
            _in_workspace(
                h.device, handle,
                lambda ws, n: _lib.linear_ce_forward(code, T, V, D, hp, ldh, wp, ldw,
                                                     targets.data_ptr(), int(ignore_index),
                                                     loss.data_ptr(), lse.data_ptr(), ws, n, handle,
                                                     check=False),
                lambda: _lib.linear_ce_workspace_bytes(code, 0, T, V, D, hp, ldh, wp, ldw),
                "gemm14_linear_ce_forward")
        return loss, lse

    return _on(stream, h.device, body)


def linear_cross_entropy_backward(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                                  lse: torch.Tensor, dloss: torch.Tensor,
                                  ignore_index: int = -100, need_dh: bool = True,
                                  need_dw: bool = True, stream=None,
                                  fp32_mode: str | None = None
                                  ) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """(dh, dw): the gradients of sum_t dloss[t] * loss[t] in h and w, in their
    dtype (gemm14_linear_ce_backward). lse: the forward call's; dloss: (T,)
    float32. Rows that take no part get zero rows in dh and add nothing to dw.
    need_dh / need_dw: a gradient not needed is not formed (None)."""
    code, T, V, D, ldh, ldw = _ce_operands(h, w, targets, fp32_mode)
    _vector(lse, "lse", T, torch.float32, h.get_device())
    _vector(dloss, "dloss", T, torch.float32, h.get_device())

    def body(handle):
        dh = torch.empty((T, D), dtype=h.dtype, device=h.device) if need_dh else None
        dw = torch.empty((V, D), dtype=w.dtype, device=w.device) if need_dw else None
        if need_dw or (need_dh and T):
            hp, wp = _ptr(h), w.data_ptr()
            _in_workspace(
                h.device, handle,
                lambda ws, n: _lib.linear_ce_backward(code, T, V, D, hp, ldh, wp, ldw, _ptr(targets),
                                                      int(ignore_index), _ptr(lse), _ptr(dloss),
                                                      _ptr(dh), D, _ptr(dw), D, ws, n, handle,
                                                      check=False),
                lambda: _lib.linear_ce_workspace_bytes(code, 1, T, V, D, hp, ldh, wp, ldw),
                "gemm14_linear_ce_backward")
        return dh, dw

    return _on(stream, h.device, body)


class Ckpt8:
    """A matrix kept in 8 bits: q (rows, cols) int8 and a scale byte for each
    block of 32 columns, scale (rows, ceil(cols / 32)) uint8; a value stands
    for q * 2**(scale - 133). Both are row-major views on one GPU; 16-byte
    aligned rows (as ckpt8_save allocates them) give the fastest accesses."""

    __slots__ = ("_q", "_scale", "_pitches")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        self._q, self._scale, self._pitches = q, scale, None

    def _operands(self) -> tuple[torch.Tensor, torch.Tensor, int, int]:
        """q, scale and their pitches, checked at their first use."""
        q, scale = self._q, self._scale
        if self._pitches is None:
            ldq = _matrix(q, "q")
            lds = _matrix(scale, "scale", q.get_device())
            rows, cols = q.shape
            if q.dtype != torch.int8 or scale.dtype != torch.uint8 or \
                    scale.shape != (rows, -(-cols // CKPT8_BLOCK)):
                raise ValueError("q must be int8 (rows, cols) and scale uint8 (rows, ceil(cols / 32)), "
                                 f"got {q.dtype} {tuple(q.shape)}, {scale.dtype} {tuple(scale.shape)}")
            self._pitches = (ldq, lds)
        return q, scale, *self._pitches

    @property
    def q(self) -> torch.Tensor:
        return self._q

    @property
    def scale(self) -> torch.Tensor:
        return self._scale

    @property
    def shape(self) -> torch.Size:
        return self._q.shape


def ckpt8_save(x: torch.Tensor, stream=None) -> Ckpt8:
    """x (rows, cols), float32, bfloat16 or float16, kept in 8 bits (gemm14_ckpt8_save)."""
    if x.dtype not in _CODE:
        raise TypeError(f"unsupported dtype {x.dtype}")
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    blocks = -(-cols // CKPT8_BLOCK)
    ldq, lds = -(-cols // 16) * 16, -(-blocks // 16) * 16

    def body(handle):
        # rows of both on 16 bytes
        q = torch.empty_strided((rows, cols), (ldq, 1), dtype=torch.int8, device=x.device)
        scale = torch.empty_strided((rows, blocks), (lds, 1), dtype=torch.uint8, device=x.device)
        if x.numel():
            _lib.ckpt8_save_raw(_CODE[x.dtype], rows, cols, x.data_ptr(), ldx, q.data_ptr(), ldq,
                                scale.data_ptr(), lds, handle)
        kept = Ckpt8(q, scale)
        kept._pitches = (max(ldq, 1), max(lds, 1))
        return kept

    return _on(stream, x.device, body)


def ckpt8_restore(c: Ckpt8, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of a checkpoint as a (rows, cols) tensor of dtype (gemm14_ckpt8_restore)."""
    if dtype not in _CODE:
        raise TypeError(f"unsupported dtype {dtype}")
    q, scale, ldq, lds = c._operands()
    rows, cols = q.shape
    device = q.device

    def body(handle):
        out = torch.empty((rows, cols), dtype=dtype, device=device)
        if out.numel():
            _lib.ckpt8_restore_raw(_CODE[dtype], rows, cols, q.data_ptr(), ldq, scale.data_ptr(),
                                   lds, out.data_ptr(), cols, handle)
        return out

    return _on(stream, device, body)


def ckpt8_weight_grad(dy: torch.Tensor, c: Ckpt8, out: torch.Tensor | None = None,
                      alpha: float = 1.0, beta: float = 0.0, stream=None,
                      fp32_mode: str | None = None) -> torch.Tensor:
    """out = alpha * dy.T @ x + beta * out, x the values of the checkpoint: the
    weight gradient of y = x @ w.T (gemm14_ckpt8_wgrad). dy: (T, N) in float32,
    bfloat16 or float16; out: (N, K) float32, row-major, allocated if not given
    (beta is then 0). beta = 1 adds to the gradient that is there."""
    code = _code(dy, fp32_mode)
    lddy = _matrix(dy, "dy")
    q, scale, ldq, lds = c._operands()
    (T, N), (T2, K) = dy.shape, q.shape
    if T != T2 or q.get_device() != dy.get_device():
        raise ValueError(f"dy {tuple(dy.shape)} and the checkpoint {tuple(q.shape)} differ in "
                         "rows or device")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
    elif out.dtype != torch.float32 or out.shape != (N, K):
        raise ValueError(f"out must be float32 of shape {(N, K)}")

    def body(handle):
        dw = out if out is not None else torch.empty((N, K), dtype=torch.float32, device=dy.device)
        lddw = _matrix(dw, "out", dy.get_device())
        if not dw.numel():
            return dw
        _in_workspace(
            dy.device, handle,
            lambda ws, n: _lib.ckpt8_wgrad(code, T, N, K, float(alpha), _ptr(dy), lddy, _ptr(q),
                                           ldq, _ptr(scale), lds, float(beta), dw.data_ptr(),
                                           lddw, ws, n, handle, check=False),
            lambda: _lib.ckpt8_wgrad_workspace_bytes(code, T, N, K, _ptr(dy), lddy, dw.data_ptr(),
                                                     lddw),
            "gemm14_ckpt8_wgrad")
        return dw

    return _on(stream, dy.device, body)


# Calls of up to this many tokens need no workspace (and no lock for it), others one.
_FEW_TOKENS = 1024


def _tokens(tokens: torch.Tensor, device: int) -> int:
    """The bytes of a token (a contiguous integer tensor on the device of this index)."""
    if tokens.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"tokens must be int64 or int32, got {tokens.dtype}")
    if tokens.get_device() != device or not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous, on the operands' device, got strides "
                         f"{tokens.stride()} on {tokens.device}")
    return tokens.element_size()


def embedding(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0,
              ignore_index: int = -100, dtype: torch.dtype | None = None,
              stream=None) -> torch.Tensor:
    """scale * table[tokens] (gemm14_embedding_forward), of shape (*tokens.shape, D).

    table: (V, D) float32, bfloat16 or float16, a row-major view; tokens: int64 or
    int32 of any shape, contiguous, on the same GPU. The row of a token that is
    ignore_index is 0, that of another outside [0, V) NaN. dtype: the output's
    (default: the table's). Stream, allocation and autograd as for
    linear_cross_entropy; embedding_backward forms the gradient."""
    dtype = table.dtype if dtype is None else dtype
    code, out_code = _CODE.get(table.dtype), _CODE.get(dtype)
    if code is None or out_code is None:
        raise TypeError(f"unsupported dtypes {table.dtype}, {dtype}")
    ldw = _matrix(table, "table")
    index = table.get_device()
    size = _tokens(tokens, index)
    if table.numel() == 0:
        raise ValueError(f"table must not be empty, got shape {tuple(table.shape)}")
    if stream is None and index == _current_device():  # (the time of a lookup of few tokens is the host's)
        return _lookup(_current_stream(index), code, out_code, table, ldw, tokens, size, ignore_index,
                       scale, dtype)
    return _on(stream, table.device,
               lambda handle: _lookup(handle, code, out_code, table, ldw, tokens, size, ignore_index,
                                      scale, dtype))


def _lookup(handle, code, out_code, table, ldw, tokens, size, ignore_index, scale, dtype):
    V, D = table.shape
    T = tokens.numel()
    out = torch.empty((*tokens.shape, D), dtype=dtype, device=table.device)
    if T:
        status = _lib.load().gemm14_embedding_forward(code, out_code, T, V, D, table.data_ptr(), ldw,
                                                      tokens.data_ptr(), size, int(ignore_index),
                                                      float(scale), out.data_ptr(), D, handle)
        if status:
            raise _lib.Gemm14Error(status, "gemm14_embedding_forward")
    return out


def embedding_backward(dy: torch.Tensor, tokens: torch.Tensor, rows: int | None = None,
                       out: torch.Tensor | None = None, scale: float = 1.0, beta: float = 0.0,
                       ignore_index: int = -100, dtype: torch.dtype | None = None,
                       stream=None) -> torch.Tensor:
    """out = scale * (the rows of dy summed by token) + beta * out: the gradient of
    embedding(table, tokens, scale) in its table (gemm14_embedding_backward).

    dy: (*tokens.shape, D) float32, bfloat16 or float16; a row-major matrix view
    where tokens has one dimension, else contiguous. out: (V, D), row-major, of
    dy's dtype or float32; or rows = V, and it is allocated, in dtype (default:
    dy's; beta is then 0). beta = 1 adds to the gradient that is there and leaves
    rows without tokens as they are: the output projection's, where the two share
    their weights. Tokens that are ignore_index or outside [0, V) add nothing. Sums
    are fp32, in an order that repeats. Stream and workspace as for
    linear_cross_entropy."""
    code = _CODE.get(dy.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dy.dtype}")
    if dy.dim() != tokens.dim() + 1 or dy.shape[:-1] != tokens.shape:
        raise ValueError(f"dy {tuple(dy.shape)} must have a row for each of the tokens {tuple(tokens.shape)}")
    if dy.dim() != 2:
        if not dy.is_contiguous():
            raise ValueError("dy must be contiguous where tokens is not one-dimensional")
        dy = dy.view(tokens.numel(), dy.size(-1))
    lddy = _matrix(dy, "dy")
    index = dy.get_device()
    size = _tokens(tokens, index)
    T, D = dy.shape
    if out is None:
        if rows is None or beta != 0.0:
            raise ValueError("rows or out is needed, and out for beta != 0")
        V, dtype, lddw = int(rows), dy.dtype if dtype is None else dtype, D
    else:
        lddw = _matrix(out, "out", index)
        if out.size(1) != D or (rows is not None and out.size(0) != rows) or \
                dtype not in (None, out.dtype):
            raise ValueError(f"out {out.dtype} {tuple(out.shape)} does not fit rows {rows}, "
                             f"{D} columns and dtype {dtype}")
        V, dtype = out.size(0), out.dtype
    if dtype not in (dy.dtype, torch.float32):
        raise TypeError(f"the gradient is formed in dy's dtype or float32, not {dtype}")
    if V < 1 or D < 1:
        raise ValueError(f"an empty table has no gradient: {V} rows of {D}")
    device, out_code = dy.device, _CODE[dtype]

    def body(handle):
        dw = out if out is not None else torch.empty((V, D), dtype=dtype, device=device)
        fn = _lib.load().gemm14_embedding_backward
        args = (code, out_code, T, V, D, _ptr(dy), lddy, _ptr(tokens), size, int(ignore_index),
                float(scale), float(beta), dw.data_ptr(), lddw)
        if T <= _FEW_TOKENS:
            status = fn(*args, None, 0, handle)
            if status:
                raise _lib.Gemm14Error(status, "gemm14_embedding_backward")
        else:
            _in_workspace(device, handle, lambda ws, n: fn(*args, ws, n, handle),
                          lambda: _lib.embedding_backward_workspace_bytes(code, T, V, D),
                          "gemm14_embedding_backward")
        return dw

    return _on(stream, device, body)


def _as_rows(x: torch.Tensor) -> tuple[int, int, int, object]:
    """(rows, cols, pitch) of a tensor's elements: a row-major matrix as it is,
    another in the order its elements lie in memory, one row where without gaps;
    and that order (equal for tensors whose elements follow one another alike)."""
    if x.numel() == 0:
        return 0, 0, 1, None
    if x.dim() == 2 and (x.size(1) == 1 or x.stride(1) == 1) and \
            (x.size(0) == 1 or x.stride(0) >= x.size(1)):
        return x.size(0), x.size(1), max(x.stride(0), x.size(1)), "rows"
    if x.is_contiguous():
        return 1, x.numel(), x.numel(), "dense"
    dims = sorted((s, n) for s, n in zip(x.stride(), x.shape) if n > 1)
    cols, rows, ld = 1, 1, 1
    while dims and dims[0][0] == cols:
        cols *= dims.pop(0)[1]
    if dims:
        ld = dims[0][0]
        for s, n in dims:
            if s != ld * rows:
                ld = 0
                break
            rows *= n
    if ld < cols and rows > 1 or ld == 0:
        raise ValueError(f"strides {x.stride()} of shape {tuple(x.shape)} are not rows of one pitch")
    return rows, cols, max(ld, cols), x.stride()


_address = torch.Tensor.data_ptr
_storage_address, _storage_bytes = torch.UntypedStorage.data_ptr, torch.UntypedStorage.nbytes


class GradList:
    """Tensors that grad_norm and clip_grad_norm take together: float32, bfloat16
    and float16 CUDA tensors of one GPU, in any mixture, each without gaps or rows
    of one pitch. A program that keeps its gradients keeps the list of them too:
    making it costs some 2.5 us a tensor, a look at it in a call 0.1 to 0.3 (109
    tensors on the GB300's host). Calls read and write the elements that the tensors
    have when the list is made. A tensor that is given other memory later (.data,
    set_, a resize of it or of its storage) needs a new list: a call on the old one
    raises ValueError."""

    __slots__ = ("_tensors", "_args", "_device", "_layouts", "_dtypes", "_storages", "_at")

    def __init__(self, tensors):
        self._tensors = tuple(tensors)
        self._args = (_lib.TensorArg * len(self._tensors))()
        self._device = None
        self._layouts, self._dtypes = [], []
        storages = {}  # each once
        for x in self._tensors:
            s = x.untyped_storage()
            storages[s._cdata] = s
        self._storages = tuple(storages.values())
        self._at = self._memory()
        for i, (x, a) in enumerate(zip(self._tensors, self._args)):
            if x.dtype not in _CODE:
                raise TypeError(f"tensor {i}: unsupported dtype {x.dtype}")
            if not x.is_cuda or (self._device is not None and x.device != self._device):
                raise ValueError(f"tensor {i} must be a CUDA tensor on the others' device, is on {x.device}")
            self._device = x.device
            a.rows, a.cols, a.ld, order = _as_rows(x)
            a.data, a.dtype = _ptr(x), _CODE[x.dtype]
            self._layouts.append((x.shape, order))
            self._dtypes.append(a.dtype)

    def _memory(self) -> list[int]:
        """Where the tensors are, and where their storages and how large: holding a
        storage keeps it from being freed, not from being resized to other memory."""
        return [*map(_address, self._tensors), *map(_storage_address, self._storages),
                *map(_storage_bytes, self._storages)]

    def _check(self) -> None:
        """Refuses the list where one of its tensors has other memory than when it was made."""
        now = self._memory()
        if now != self._at:
            i = next(i for i, (a, b) in enumerate(zip(now, self._at)) if a != b)
            what = f"tensor {i}" if i < len(self._tensors) else "a tensor's storage"
            raise ValueError(f"{what} has been given other memory since the list was made: make a "
                             "new GradList")

    @property
    def tensors(self) -> tuple[torch.Tensor, ...]:
        return self._tensors

    def __len__(self) -> int:
        return len(self._tensors)


def _list_of(tensors) -> GradList:
    """The list that a call is given, or that of its tensors."""
    if not isinstance(tensors, GradList):
        return GradList(tensors)
    tensors._check()
    return tensors


def _grad_call(grads, each, stream, call, where):
    """The norm, or it and each, of call(norm, each, workspace, bytes, stream handle)."""
    device = grads._device or torch.device("cuda", torch.cuda.current_device())
    n = len(grads._tensors)

    def body(handle):
        norm = torch.empty((), dtype=torch.float32, device=device)
        norms = torch.empty(n, dtype=torch.float32, device=device) if each else None
        at, each_at = norm.data_ptr(), _ptr(norms)
        try:
            _in_workspace(device, handle, lambda ws, b: call(at, each_at, ws, b, handle),
                          lambda: _lib.grad_workspace_bytes(n), where)
        except _lib.Gemm14Error as e:
            if e.status == _lib.GEMM14_ERR_INVALID_ARG:
                raise ValueError(f"{where}: {_lib.last_error_string()}") from e
            raise
        return (norm, norms) if each else norm

    return _on(stream, device, body)


def grad_norm(grads, scale: float = 1.0, each: bool = False, stream=None):
    """|scale| * the square root of the sum of the squares of all elements of all of
    grads (a GradList or a sequence of tensors), a 0-dimensional float32 tensor on
    their GPU; with each, also the norm of each of them, a float32 vector
    (gemm14_grad_norm). scale: 1 / the loss scale. Sums are held in fp64 and
    repeat. Stream and workspace as for linear_cross_entropy."""
    grads = _list_of(grads)
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    n, args, scale = len(grads._tensors), grads._args, float(scale)
    fn = _lib.load().gemm14_grad_norm
    return _grad_call(grads, each, stream,
                      lambda norm, norms, ws, b, handle: fn(n, args, scale, norm, norms, ws, b, handle),
                      "gemm14_grad_norm")


def clip_grad_norm(grads, max_norm: float, scale: float = 1.0, out=None, each: bool = False,
                   stream=None):
    """Scales grads (a GradList or a sequence of tensors) by scale * min(1, max_norm
    / norm), in place or into out (as many tensors of the same shapes and strides,
    each of its gradient's dtype or float32), and returns the norm, as grad_norm
    does, of before (gemm14_grad_clip). scale takes gradients out of a loss scale. Where
    an element is infinite or NaN, so is the norm, and nothing is clipped: out =
    scale * grads, for the caller to leave alone. Finite elements are clipped always,
    also where their norm is beyond float32's largest number and so returned as
    infinite. No tensor that is written may share memory with another of the
    lists. Nothing is copied to the host."""
    grads = _list_of(grads)
    if out is not None:
        out = _list_of(out)
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    if not max_norm >= 0.0:
        raise ValueError(f"max_norm must not be negative, got {max_norm}")
    if out is not None:
        if len(out) != len(grads) or (len(out) and out._device != grads._device):
            raise ValueError(f"{len(grads)} gradients and {len(out)} outputs, on one device each")
        if grads._layouts != out._layouts or \
                (grads._dtypes != out._dtypes and any(out._dtypes)):  # (0 is float32)
            for i, (x, y) in enumerate(zip(grads._tensors, out._tensors)):
                if y.dtype not in (x.dtype, torch.float32) or grads._layouts[i] != out._layouts[i]:
                    raise ValueError(f"output {i} ({y.dtype} {tuple(y.shape)}, strides {y.stride()}) "
                                     f"does not fit its gradient ({x.dtype} {tuple(x.shape)}, "
                                     f"{x.stride()})")
    n, args, out_args = len(grads._tensors), grads._args, None if out is None else out._args
    scale, max_norm = float(scale), float(max_norm)
    fn = _lib.load().gemm14_grad_clip
    return _grad_call(grads, each, stream,
                      lambda norm, norms, ws, b, handle: fn(n, args, out_args, scale, max_norm, norm,
                                                            norms, ws, b, handle),
                      "gemm14_grad_clip")
