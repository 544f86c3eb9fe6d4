"""The loss of a linear head against a teacher's top logits, and its gradients.

Distillation: tau^2 KL(teacher || student) at temperature tau over the entries
that the teacher kept of each row, with the student's logits formed tile by
tile as the cross entropy's are (the kernels: csrc/distill.cu, csrc/loss.cu,
csrc/loss_gemm.cuh). In a training step of sharded units the weight is a view
of a unit's gathered buffer and d_weight a view of a rank's flat gradient
buffer ("Data Parallelism", "The Basic Protocol").
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from .fsdp import _check, _counter, dtype_code
from .loss import _REDUCTIONS, Head, _matrix, _refuse_device, _vector
from .workspace import take

__all__ = ["HeadDistill", "fsdp_head_distill"]

_ID_BITS = {torch.int32: 32, torch.int64: 64}


def _blank(temperature: float, reduction: str, band: int) -> _lib.FsdpHeadDistillArgs:
    """A call's arguments that do not change from one to the next."""
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTIONS)}")
    a = _lib.FsdpHeadDistillArgs()
    a.temperature, a.reduction, a.band, a.grad_scale = float(temperature), _REDUCTIONS[reduction], int(band), 1.0
    return a


def _fill(a: _lib.FsdpHeadDistillArgs, hidden, weight, teacher_logits, teacher_ids, loss, token_loss, d_hidden, d_weight,
          grad_scale, wait_timeouts) -> int:
    """The tensors of a call; the device."""
    for t, name in ((hidden, "hidden"), (weight, "weight"), (teacher_logits, "teacher_logits"),
                    (teacher_ids, "teacher_ids")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a matrix")
    if teacher_ids.dtype not in _ID_BITS:
        raise ValueError("teacher_ids must be int32 or int64")
    if not hidden.is_cuda:
        _refuse_device(hidden, "hidden")
    cur = torch.cuda.current_device()
    T, D = hidden.shape
    V, K = weight.shape[0], teacher_ids.shape[1]
    dt, tdt = hidden.dtype, teacher_logits.dtype
    a.dtype, a.teacher_dtype, a.id_bits = dtype_code(dt), dtype_code(tdt), _ID_BITS[teacher_ids.dtype]
    a.tokens, a.vocab, a.dim, a.top = T, V, D, K
    a.hidden, a.ld_hidden = _matrix(hidden, "hidden", T, D, dt, cur)
    a.weight, a.ld_weight = _matrix(weight, "weight", V, D, dt, cur)
    a.teacher_logits, a.ld_teacher_logits = _matrix(teacher_logits, "teacher_logits", T, K, tdt, cur)
    a.teacher_ids, a.ld_teacher_ids = _matrix(teacher_ids, "teacher_ids", T, K, teacher_ids.dtype, cur)
    a.loss = _vector(loss, "loss", 1, torch.float32, cur)
    if token_loss is not None:
        a.token_loss = _vector(token_loss, "token_loss", T, torch.float32, cur)
    if d_hidden is not None:
        a.d_hidden, a.ld_d_hidden = _matrix(d_hidden, "d_hidden", T, D, dt, cur)
    if d_weight is not None:
        a.d_weight, a.ld_d_weight = _matrix(d_weight, "d_weight", V, D, dt, cur)
    a.grad_scale = float(grad_scale)
    if wait_timeouts is not None:
        a.wait_timeouts = _counter(wait_timeouts, "wait_timeouts")
    return cur


def _workspace_bytes(a: _lib.FsdpHeadDistillArgs) -> int:
    n = ctypes.c_int64(0)
    _check(_lib.load().fsdp_head_distill_workspace(ctypes.byref(a), ctypes.byref(n)), "fsdp_head_distill_workspace")
    return int(n.value)


def fsdp_head_distill(hidden: torch.Tensor, weight: torch.Tensor, teacher_logits: torch.Tensor,
                      teacher_ids: torch.Tensor, loss: torch.Tensor, token_loss: Optional[torch.Tensor] = None,
                      d_hidden: Optional[torch.Tensor] = None, d_weight: Optional[torch.Tensor] = None,
                      temperature: float = 1.0, reduction: str = "mean", grad_scale: float = 1.0, band: int = 0,
                      wait_timeouts: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """The C entry point with a workspace of its own for this one call.

    hidden [T, D], weight [V, D] (rows contiguous, any stride and alignment),
    teacher_logits [T, K] of fp32, bf16 or fp16 and teacher_ids [T, K] of int32
    or int64 (rows contiguous; -1: no entry); loss fp32 scalar, token_loss fp32
    [T], d_hidden [T, D] and d_weight [V, D] of hidden's dtype are written (d_*
    None: not formed)."""
    a = _blank(temperature, reduction, band)
    _fill(a, hidden, weight, teacher_logits, teacher_ids, loss, token_loss, d_hidden, d_weight, grad_scale, wait_timeouts)
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.stream(s):  # taken, and given back, in that stream's order
        ws = take(_workspace_bytes(a), hidden.device, alignment=1024)
    _check(_lib.load().fsdp_head_distill(ctypes.byref(a), ws.data_ptr(), ws.numel(), s.cuda_stream),
           "fsdp_head_distill")


class HeadDistill(Head):
    """A head's distillation loss with the workspace its calls share.

    vocab, dim, dtype: the weight's shape and the dtype of hidden, weight and
    gradients. max_tokens: the most rows of a call; top: the most entries that
    the teacher has of a row (at most 1024). temperature: what both sides'
    logits are divided by. grad, band, reduction ("mean" over the rows that have
    an entry, or "sum") and the workspace as in HeadLoss. Calls on one stream,
    or ordered between streams, may share the object; calls that run at the
    same time need a HeadDistill each."""

    def __init__(self, vocab: int, dim: int, dtype: torch.dtype, max_tokens: int, top: int, temperature: float = 1.0,
                 grad: bool = True, band: int = 0, reduction: str = "mean", device="cuda"):
        self.top, self.temperature = int(top), float(temperature)
        self._blank = _blank(temperature, reduction, band)
        self._start(vocab, dim, dtype, max_tokens, grad, band, reduction, device)

    def _sized(self, step: int) -> _lib.FsdpHeadDistillArgs:
        a = _lib.FsdpHeadDistillArgs.from_buffer_copy(self._blank)
        a.teacher_logits, a.teacher_ids = 3 * step, 7 * step
        a.top = a.ld_teacher_logits = a.ld_teacher_ids = self.top
        a.teacher_dtype, a.id_bits = _lib.FSDP_F32, 64
        return a

    def _bytes(self, a: _lib.FsdpHeadDistillArgs) -> int:
        return _workspace_bytes(a)

    def _enqueue(self, a: _lib.FsdpHeadDistillArgs, stream: int) -> int:
        return _lib.load().fsdp_head_distill(ctypes.byref(a), self._ws_at, self._ws_bytes, stream)

    def forward(self, hidden: torch.Tensor, weight: torch.Tensor, teacher_logits: torch.Tensor,
                teacher_ids: torch.Tensor, loss: Optional[torch.Tensor] = None,
                token_loss: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                wait_timeouts: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The loss (fp32 scalar) and the rows' losses (fp32 [T], 0 for a row
        without entries). loss / token_loss: where to write them (new ones
        otherwise)."""
        return self._run(hidden, weight, teacher_logits, teacher_ids, None, None, 1.0, loss, token_loss, stream,
                         wait_timeouts)

    def forward_backward(self, hidden: torch.Tensor, weight: torch.Tensor, teacher_logits: torch.Tensor,
                         teacher_ids: torch.Tensor, d_hidden: Optional[torch.Tensor],
                         d_weight: Optional[torch.Tensor], grad_scale: float = 1.0,
                         loss: Optional[torch.Tensor] = None, token_loss: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None,
                         wait_timeouts: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """forward(), and the gradients of grad_scale * loss written to
        d_hidden [T, D] and d_weight [V, D] (None: not formed)."""
        return self._run(hidden, weight, teacher_logits, teacher_ids, d_hidden, d_weight, grad_scale, loss, token_loss,
                         stream, wait_timeouts)

    def _run(self, hidden, weight, teacher_logits, teacher_ids, d_hidden, d_weight, grad_scale, loss, token_loss, stream,
             wait_timeouts):
        self._check_operands(hidden, weight)
        if not isinstance(teacher_ids, torch.Tensor) or teacher_ids.dim() != 2 or teacher_ids.shape[1] > self.top:
            raise ValueError(f"teacher_ids must be [{hidden.shape[0]}, at most {self.top}]")
        loss, token_loss = self._results(hidden, loss, token_loss, stream)
        a = _lib.FsdpHeadDistillArgs.from_buffer_copy(self._blank)
        device = _fill(a, hidden, weight, teacher_logits, teacher_ids, loss, token_loss, d_hidden, d_weight, grad_scale,
                       wait_timeouts)
        self._launch(a, stream, device, "fsdp_head_distill")
        return loss, token_loss
