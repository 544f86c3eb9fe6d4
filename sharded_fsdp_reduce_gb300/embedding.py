"""The token embedding and its gradient (the kernels: csrc/embed.cu,
csrc/embed_grad.cu).

In a training step of sharded units the table is a view of a unit's gathered
buffer and its gradient a view of a rank's flat gradient buffer; a table tied
to the head adds to the gradient that the head's loss left there ("Data
Parallelism", "The Basic Protocol").
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from .fsdp import _check, dtype_code
from .loss import _matrix, _refuse_device, _vector
from .workspace import Workspace, raw_stream, take

__all__ = ["Embedding", "fsdp_embed", "fsdp_embed_grad"]


def _matrices(*named) -> None:
    for t, name in named:
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a matrix")


def _blank(kind, vocab: int, dim: int, dtype: torch.dtype, scale: float, ignore_index: int):
    """A call's arguments that do not change from one to the next."""
    a = kind()
    a.dtype, a.vocab, a.dim = dtype_code(dtype), vocab, dim
    a.scale, a.ignore_index = float(scale), int(ignore_index)
    return a


def _fill(a, tokens, weight, out, dtype: torch.dtype, device: int) -> None:
    if not isinstance(tokens, torch.Tensor):
        _refuse_device(tokens, "tokens")
    a.count = n = tokens.numel()
    a.tokens = _vector(tokens, "tokens", n, torch.int64, device)
    a.weight, a.ld_weight = _matrix(weight, "weight", a.vocab, a.dim, dtype, device)
    a.out, a.ld_out = _matrix(out, "out", n, a.dim, dtype, device)


def _fill_grad(a, tokens, d_out, d_weight, accumulate, dtype: torch.dtype, device: int) -> None:
    if not isinstance(tokens, torch.Tensor):
        _refuse_device(tokens, "tokens")
    a.count = n = tokens.numel()
    a.tokens = _vector(tokens, "tokens", n, torch.int64, device)
    a.d_out, a.ld_d_out = _matrix(d_out, "d_out", n, a.dim, dtype, device)
    a.d_weight, a.ld_d_weight = _matrix(d_weight, "d_weight", a.vocab, a.dim, dtype, device)
    a.accumulate = 1 if accumulate else 0


def _grad_args(tokens, d_out, d_weight, scale, ignore_index, accumulate) -> _lib.FsdpEmbedGradArgs:
    _matrices((d_out, "d_out"), (d_weight, "d_weight"))
    a = _blank(_lib.FsdpEmbedGradArgs, *d_weight.shape, d_weight.dtype, scale, ignore_index)
    _fill_grad(a, tokens, d_out, d_weight, accumulate, d_weight.dtype, torch.cuda.current_device())
    return a


def _workspace_bytes(a: _lib.FsdpEmbedGradArgs) -> int:
    n = ctypes.c_int64(0)
    _check(_lib.load().fsdp_embed_grad_workspace(ctypes.byref(a), ctypes.byref(n)), "fsdp_embed_grad_workspace")
    return int(n.value)


def fsdp_embed(tokens: torch.Tensor, weight: torch.Tensor, out: torch.Tensor, scale: float = 1.0,
               ignore_index: int = -100, stream: Optional[torch.cuda.Stream] = None) -> None:
    """The C entry point: out[t] = scale * weight[tokens[t]].

    tokens int64 (any shape, contiguous; T of them), weight [V, D] and out
    [T, D] of its dtype (rows contiguous, any stride and alignment)."""
    _matrices((weight, "weight"), (out, "out"))
    a = _blank(_lib.FsdpEmbedArgs, *weight.shape, weight.dtype, scale, ignore_index)
    _fill(a, tokens, weight, out, weight.dtype, torch.cuda.current_device())
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(_lib.load().fsdp_embed(ctypes.byref(a), s.cuda_stream), "fsdp_embed")


def fsdp_embed_grad(tokens: torch.Tensor, d_out: torch.Tensor, d_weight: torch.Tensor, scale: float = 1.0,
                    ignore_index: int = -100, accumulate: bool = False,
                    stream: Optional[torch.cuda.Stream] = None) -> None:
    """The C entry point with a workspace of its own for this one call:
    d_weight [V, D] gets the table's gradient from d_out [T, D], or has it
    added (accumulate)."""
    a = _grad_args(tokens, d_out, d_weight, scale, ignore_index, accumulate)
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.stream(s):  # taken, and given back, in that stream's order
        ws = take(_workspace_bytes(a), d_weight.device)
    _check(_lib.load().fsdp_embed_grad(ctypes.byref(a), ws.data_ptr(), ws.numel(), s.cuda_stream), "fsdp_embed_grad")


class Embedding:
    """A model's token table with the workspace its gradient's calls share.

    vocab, dim, dtype: the table's shape and the dtype of it, its rows and their
    gradients. max_tokens: the most tokens of a call. scale: what rows are
    multiplied by (sqrt(dim) in some models). ignore_index: the padding, whose
    rows are zeros and which has no gradient. grad: whether backward() will be
    called (the workspace is for it). Calls on one stream, or ordered between
    streams, may share the object; backward() calls that run at the same time
    need an Embedding each."""

    def __init__(self, vocab: int, dim: int, dtype: torch.dtype, max_tokens: int, scale: float = 1.0,
                 ignore_index: int = -100, grad: bool = True, device="cuda"):
        self.vocab, self.dim, self.dtype = int(vocab), int(dim), dtype
        self.max_tokens, self.scale, self.ignore_index = int(max_tokens), float(scale), int(ignore_index)
        self.device = torch.device(device)
        self._lookup = _blank(_lib.FsdpEmbedArgs, self.vocab, self.dim, dtype, self.scale, self.ignore_index)
        self._grad = _blank(_lib.FsdpEmbedGradArgs, self.vocab, self.dim, dtype, self.scale, self.ignore_index)
        a = _lib.FsdpEmbedGradArgs.from_buffer_copy(self._grad)
        a.count = self.max_tokens
        step = 1 << 56  # (addresses are not read)
        a.tokens, a.d_out, a.d_weight = step, 2 * step, 3 * step
        a.ld_d_out = a.ld_d_weight = self.dim
        need = _workspace_bytes(a)  # checks the sizes too
        self._ws = Workspace(need, self.device) if grad else None
        self._ws_at, self._ws_bytes = (self._ws.buf.data_ptr(), need) if grad else (0, 0)

    def _check(self, tokens) -> None:
        if not isinstance(tokens, torch.Tensor) or tokens.numel() > self.max_tokens:
            raise ValueError(f"tokens must hold at most {self.max_tokens}")

    def forward(self, tokens: torch.Tensor, weight: torch.Tensor, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """scale * weight[tokens], [T, dim]: written to out, or to a new tensor."""
        self._check(tokens)
        device = torch.cuda.current_device()
        if out is None:
            with torch.cuda.stream(stream):  # a new result belongs to the call's stream
                out = torch.empty(tokens.numel(), self.dim, dtype=self.dtype, device=tokens.device)
        a = _lib.FsdpEmbedArgs.from_buffer_copy(self._lookup)
        _fill(a, tokens, weight, out, self.dtype, device)
        _check(_lib.load().fsdp_embed(ctypes.byref(a), raw_stream(stream, device)), "fsdp_embed")
        return out

    def backward(self, tokens: torch.Tensor, d_out: torch.Tensor, d_weight: torch.Tensor, accumulate: bool = False,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """The table's gradient from its rows' ([T, dim]), written to d_weight
        whole (zeros where no token points), or added to what it holds
        (accumulate: a table tied to the head, after the head's gradient)."""
        self._check(tokens)
        if self._ws is None:
            raise ValueError("this Embedding was made without gradients (grad=False)")
        device = torch.cuda.current_device()
        a = _lib.FsdpEmbedGradArgs.from_buffer_copy(self._grad)
        _fill_grad(a, tokens, d_out, d_weight, accumulate, self.dtype, device)
        raw = self._ws.enter(stream, device)
        _check(_lib.load().fsdp_embed_grad(ctypes.byref(a), self._ws_at, self._ws_bytes, raw), "fsdp_embed_grad")
        return d_weight
