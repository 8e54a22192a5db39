"""Tensor-level calls of the training products: softmax cross entropy over a
projection's outputs, and activations kept in 8 bits (argument marshalling
only; every step runs in the library's CUDA kernels). None of them is recorded
by autograd."""
from __future__ import annotations

import torch

from . import _lib
from .api import (_CODE, _FP32_MODES, _capturing, _graph_workspace, _workspace, _workspace_lock,
                  _workspaces)

_current_stream = torch._C._cuda_getCurrentRawStream

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
        if device.index == torch.cuda.current_device():
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
