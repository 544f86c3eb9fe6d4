"""The loss of a linear head over a large vocabulary, and its gradients.

Softmax cross entropy of logits = hidden @ weight.T against target tokens,
with the logits formed tile by tile and never stored in fp32 (the kernels:
csrc/loss.cu, csrc/loss_gemm.cuh). In a training step of sharded units the
weight is a view of a unit's gathered buffer and d_weight a view of a rank's
flat gradient buffer, so the gradient lands where the reduce-scatter reads it
("Data Parallelism", "The Basic Protocol").
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from .fsdp import _check, _counter, _on_current_device, dtype_code
from .workspace import Workspace, take

__all__ = ["HeadLoss", "fsdp_head_loss", "fsdp_check_head_loss_wait"]

_REDUCTIONS = {"mean": _lib.FSDP_LOSS_MEAN, "sum": _lib.FSDP_LOSS_SUM}


def _matrix(t: torch.Tensor, name: str, rows: int, cols: int, dtype: torch.dtype, device: int) -> Tuple[int, int]:
    """Address and row stride of a [rows, cols] matrix on the current device whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _refuse_device(t, name)
    if t.dtype != dtype or t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}] of {dtype}")
    stride = t.stride()
    ld = stride[0] if rows > 1 else cols
    if (cols > 1 and rows > 0 and stride[1] != 1) or ld < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld


def _vector(t: torch.Tensor, name: str, numel: int, dtype: torch.dtype, device: int) -> int:
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _refuse_device(t, name)
    if t.dtype != dtype or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must hold {numel} contiguous elements of {dtype}")
    return t.data_ptr()


def _refuse_device(t, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _on_current_device(t, name)


def _args(hidden, weight, targets, loss, token_loss, d_hidden, d_weight, ignore_index, reduction, grad_scale, band,
          wait_timeouts) -> _lib.FsdpHeadLossArgs:
    if not isinstance(hidden, torch.Tensor) or hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden and weight must be matrices")
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTIONS)}")
    T, D = hidden.shape
    V = weight.shape[0]
    dt = hidden.dtype
    if not hidden.is_cuda:
        _refuse_device(hidden, "hidden")
    cur = torch.cuda.current_device()
    a = _lib.FsdpHeadLossArgs()
    a.dtype = dtype_code(dt)
    a.tokens, a.vocab, a.dim = T, V, D
    a.hidden, a.ld_hidden = _matrix(hidden, "hidden", T, D, dt, cur)
    a.weight, a.ld_weight = _matrix(weight, "weight", V, D, dt, cur)
    a.targets = _vector(targets, "targets", T, torch.int64, cur)
    a.loss = _vector(loss, "loss", 1, torch.float32, cur)
    if token_loss is not None:
        a.token_loss = _vector(token_loss, "token_loss", T, torch.float32, cur)
    if d_hidden is not None:
        a.d_hidden, a.ld_d_hidden = _matrix(d_hidden, "d_hidden", T, D, dt, cur)
    if d_weight is not None:
        a.d_weight, a.ld_d_weight = _matrix(d_weight, "d_weight", V, D, dt, cur)
    a.ignore_index = int(ignore_index)
    a.reduction = _REDUCTIONS[reduction]
    a.grad_scale = float(grad_scale)
    a.band = int(band)
    if wait_timeouts is not None:
        a.wait_timeouts = _counter(wait_timeouts, "wait_timeouts")
    return a


def _workspace_bytes(a: _lib.FsdpHeadLossArgs) -> int:
    n = ctypes.c_int64(0)
    _check(_lib.load().fsdp_head_loss_workspace(ctypes.byref(a), ctypes.byref(n)), "fsdp_head_loss_workspace")
    return int(n.value)


def _workspace(nbytes: int, device) -> torch.Tensor:
    return take(nbytes, device, alignment=1024)


def _launch(a: _lib.FsdpHeadLossArgs, address: int, nbytes: int, stream: torch.cuda.Stream) -> int:
    return _lib.load().fsdp_head_loss(ctypes.byref(a), address, nbytes, stream.cuda_stream)


def fsdp_head_loss(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, loss: torch.Tensor,
                   token_loss: Optional[torch.Tensor] = None, d_hidden: Optional[torch.Tensor] = None,
                   d_weight: Optional[torch.Tensor] = None, ignore_index: int = -100, reduction: str = "mean",
                   grad_scale: float = 1.0, band: int = 0, wait_timeouts: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """The C entry point with a workspace of its own for this one call.

    hidden [T, D], weight [V, D] (rows contiguous, any stride and alignment),
    targets int64 [T]; loss fp32 scalar, token_loss fp32 [T], d_hidden [T, D]
    and d_weight [V, D] of hidden's dtype are written (d_* None: not formed)."""
    a = _args(hidden, weight, targets, loss, token_loss, d_hidden, d_weight, ignore_index, reduction, grad_scale,
              band, wait_timeouts)
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.stream(s):  # taken, and given back, in that stream's order
        ws = _workspace(_workspace_bytes(a), hidden.device)
    _check(_launch(a, ws.data_ptr(), ws.numel(), s), "fsdp_head_loss")


def fsdp_check_head_loss_wait(limit_cycles: int, arrive_after_cycles: int, outcomes: torch.Tensor,
                              wait_timeouts: Optional[torch.Tensor] = None,
                              stream: Optional[torch.cuda.Stream] = None) -> None:
    """Self-test of the matrix products' bounded wait (see include/fsdp.h):
    outcomes (int32 [128]) gets 1 per thread whose wait saw the arrival."""
    at = _vector(outcomes, "outcomes", 128, torch.int32, torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(_lib.load().fsdp_check_head_loss_wait(int(limit_cycles), int(arrive_after_cycles), at,
                                                 _counter(wait_timeouts, "wait_timeouts"), s.cuda_stream),
           "fsdp_check_head_loss_wait")


class HeadLoss:
    """A head's loss with the workspace its calls share.

    vocab, dim, dtype: the weight's shape and the dtype of hidden, weight and
    gradients. max_tokens: the most rows of a call. grad: whether gradients
    will be asked for (the workspace is sized for it). band: rows worked on
    together (0: as many as keep the 16-bit exponentials within 4 GiB).
    ignore_index, reduction ("mean" over the rows that count, or "sum") as in
    fsdp_head_loss. No call of up to max_tokens rows, contiguous or 16-byte
    aligned, needs more workspace than the object starts with. Other rows of
    16-bit types are packed into it, and gradients of an object made without
    them need more: the first such call takes a larger one, and the earlier one
    is kept, so that a captured graph of earlier calls still finds it. Calls on one stream,
    or ordered between streams, may share the object; calls that run at the
    same time need a HeadLoss each."""

    def __init__(self, vocab: int, dim: int, dtype: torch.dtype, max_tokens: int, grad: bool = True, band: int = 0,
                 ignore_index: int = -100, reduction: str = "mean", device="cuda"):
        if reduction not in _REDUCTIONS:
            raise ValueError(f"reduction must be one of {sorted(_REDUCTIONS)}")
        self.vocab, self.dim, self.dtype = int(vocab), int(dim), dtype
        self.max_tokens, self.grad, self.band = int(max_tokens), bool(grad), int(band)
        self.ignore_index, self.reduction = int(ignore_index), reduction
        self.device = torch.device(device)
        self._kept = []
        odd = self.dim % 8 != 0  # (contiguous rows are then not aligned)
        self._forms = (self.grad, odd, odd)
        self._allocate(self._need(*self._forms))

    def _need(self, grad: bool, odd_hidden: bool, odd_weight: bool) -> int:
        """Workspace of every call of up to max_tokens rows: with gradients or
        not, hidden and weight 16-byte aligned or not (addresses are not read)."""
        a = _lib.FsdpHeadLossArgs()
        a.dtype = dtype_code(self.dtype)
        a.tokens, a.vocab, a.dim, a.band = self.max_tokens, self.vocab, self.dim, self.band
        step, off = 1 << 56, self.dtype.itemsize
        a.hidden, a.weight = step + (off if odd_hidden else 0), 2 * step + (off if odd_weight else 0)
        a.targets, a.loss = 3 * step, 4 * step
        a.ld_hidden = a.ld_weight = a.ld_d_hidden = a.ld_d_weight = -(-self.dim // 8) * 8
        a.grad_scale = 1.0
        need = _workspace_bytes(a)
        if grad:
            a.d_hidden, a.d_weight = 5 * step, 6 * step
            need = max(need, _workspace_bytes(a))
        return need

    def _allocate(self, nbytes: int) -> None:
        self._ws = Workspace(nbytes, self.device, alignment=1024)
        self._ws_at, self._ws_bytes = self._ws.buf.data_ptr(), nbytes

    def _grow(self, a: _lib.FsdpHeadLossArgs) -> None:
        """A larger workspace, for a call's form and all the earlier ones."""
        odd = [p % 16 != 0 or ld % 8 != 0 for p, ld in ((a.hidden, a.ld_hidden), (a.weight, a.ld_weight))]
        new = (a.d_hidden is not None or a.d_weight is not None, *odd)
        self._forms = tuple(x or y for x, y in zip(self._forms, new))
        self._kept.append(self._ws)
        self._allocate(self._need(*self._forms))

    def forward(self, hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                loss: Optional[torch.Tensor] = None, token_loss: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None,
                wait_timeouts: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The loss (fp32 scalar) and the tokens' losses (fp32 [T], 0 where
        ignored). loss / token_loss: where to write them (new ones otherwise)."""
        return self._run(hidden, weight, targets, None, None, 1.0, loss, token_loss, stream, wait_timeouts)

    def forward_backward(self, hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                         d_hidden: Optional[torch.Tensor], d_weight: Optional[torch.Tensor], grad_scale: float = 1.0,
                         loss: Optional[torch.Tensor] = None, token_loss: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None,
                         wait_timeouts: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """forward(), and the gradients of grad_scale * loss written to
        d_hidden [T, D] and d_weight [V, D] (None: not formed)."""
        return self._run(hidden, weight, targets, d_hidden, d_weight, grad_scale, loss, token_loss, stream,
                         wait_timeouts)

    def _run(self, hidden, weight, targets, d_hidden, d_weight, grad_scale, loss, token_loss, stream, wait_timeouts):
        if hidden.dim() != 2 or hidden.shape[0] > self.max_tokens or hidden.shape[1] != self.dim:
            raise ValueError(f"hidden must be [at most {self.max_tokens}, {self.dim}]")
        if hidden.dtype != self.dtype or tuple(weight.shape) != (self.vocab, self.dim):
            raise ValueError(f"hidden must be {self.dtype} and weight [{self.vocab}, {self.dim}]")
        s = stream if stream is not None else torch.cuda.current_stream()
        if loss is None or token_loss is None:
            with torch.cuda.stream(s):  # new results belong to the call's stream
                if loss is None:
                    loss = torch.empty((), dtype=torch.float32, device=hidden.device)
                if token_loss is None:
                    token_loss = torch.empty(hidden.shape[0], dtype=torch.float32, device=hidden.device)
        a = _args(hidden, weight, targets, loss, token_loss, d_hidden, d_weight, self.ignore_index, self.reduction,
                  grad_scale, self.band, wait_timeouts)
        self._ws.on(s)
        status = _launch(a, self._ws_at, self._ws_bytes, s)
        if status == _lib.FSDP_ERR_INVALID_ARG and _workspace_bytes(a) > self._ws_bytes:
            with torch.cuda.stream(s):
                self._grow(a)
            status = _launch(a, self._ws_at, self._ws_bytes, s)
        _check(status, "fsdp_head_loss")
        return loss, token_loss
