"""The global gradient norm and clipping: over a list of tensors, and inside a
model's step (the kernels: csrc/clip_norm.cu, csrc/clip_scale.cu,
csrc/clip_update.cuh)."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from .fsdp import StepConfig, UnitDescs, _check, _counter, _dev, dtype_code
from .workspace import Workspace

__all__ = ["GradClip", "ClipPlan"]


def _scalar(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() != 1:
        raise ValueError(f"{name} must be a float32 CUDA scalar")
    return _dev(t, name)


class GradClip:
    """The L2 norm over gradient tensors and their scaling to a largest norm.

    tensors: contiguous CUDA tensors of fp32, bf16 or fp16 (mixed is fine).
    out: where clip() writes (same sizes and dtypes, any alignment, e.g. the
    parameters' views of a rank's flat gradient buffer); default: in place.
    scale: what the gradients are multiplied by, the inverse of a loss scale
    they carry. Holds the tensors and their addresses: build a new one when
    a tensor is replaced. Calls on one stream, or ordered between streams."""

    def __init__(self, tensors: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None,
                 scale: float = 1.0):
        self.tensors = list(tensors)
        self.out = self.tensors if out is None else list(out)
        self.scale = float(scale)
        n = len(self.tensors)
        if len(self.out) != n:
            raise ValueError(f"out must hold {n} tensors")
        for i, (t, o) in enumerate(zip(self.tensors, self.out)):
            if o.dtype != t.dtype or o.numel() != t.numel():
                raise ValueError(f"out[{i}] must hold {t.numel()} elements of {t.dtype}")
        self._src = (ctypes.c_void_p * max(n, 1))(*[_dev(t, f"tensors[{i}]") for i, t in enumerate(self.tensors)])
        self._dst = (ctypes.c_void_p * max(n, 1))(*[_dev(t, f"out[{i}]") for i, t in enumerate(self.out)])
        self._numels = (ctypes.c_int64 * max(n, 1))(*[t.numel() for t in self.tensors])
        self._dtypes = (ctypes.c_int32 * max(n, 1))(*[dtype_code(t.dtype) for t in self.tensors])
        self._n = n
        size = ctypes.c_int64(0)
        _check(_lib.load().fsdp_grad_norm_workspace(self._numels, self._dtypes, n, ctypes.byref(size)),
               "fsdp_grad_norm_workspace")
        device = self.tensors[0].device if n else torch.device("cuda", torch.cuda.current_device())
        # the norm lies behind the kernels' part, so that a stream that is ordered
        # after the workspace's zeroing, and holds it, does so for both
        at = -(-size.value // 256) * 256
        self._ws = Workspace(at + 4, device, zeroed=True)
        self._norm = self._ws.buf[at:].view(torch.float32).reshape(())

    def norm(self, out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """The norm of scale * tensors, an fp32 CUDA scalar: out, or one this
        object keeps and overwrites with every call."""
        norm = self._norm if out is None else out
        s = self._ws.on(stream)
        _check(_lib.load().fsdp_grad_norm(self._src, self._numels, self._dtypes, self._n, self.scale,
                                          _scalar(norm, "out"), self._ws.buf.data_ptr(), self._ws.buf.numel(),
                                          s.cuda_stream), "fsdp_grad_norm")
        return norm

    def clip(self, max_norm: float, norm: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """out = tensors * scale * min(1, max_norm / (norm + 1e-6)). norm: the
        norm to use (a CUDA scalar, e.g. one taken over more tensors than
        these); default: these tensors', taken first. Returns the norm."""
        self._ws.check_device()
        s = stream if stream is not None else torch.cuda.current_stream()
        if norm is None:
            norm = self.norm(stream=s)
        _check(_lib.load().fsdp_clip_grads(self._src, self._dst, self._numels, self._dtypes, self._n,
                                           _scalar(norm, "norm"), float(max_norm), self.scale, s.cuda_stream),
               "fsdp_clip_grads")
        return norm


class ClipPlan:
    """A model's clipped step, validated once (fsdp_clip_plan_create, or
    fsdp_clip_plan_create_ex when `config` is given): launch() takes the
    averaged gradient's norm over all units, then each unit's step with the
    clipped gradient and its all-gathers. The units' buffers must stay
    allocated (the units are kept alive here). workspace: another plan's, to
    work in where it is large enough (their launches then have to be in order)."""

    def __init__(self, units, gathers: int = 1, nonfinite_count: Optional[torch.Tensor] = None,
                 config: Optional[StepConfig] = None, wait_timeouts: Optional[torch.Tensor] = None,
                 workspace: Optional[Workspace] = None):
        self.descs = units if isinstance(units, UnitDescs) else UnitDescs(units)
        if config is None and not self.descs.adamw:
            raise ValueError("an AdamW model step needs fp32 master and AdamW state in every unit")
        self.config = config
        self._counters = (nonfinite_count, wait_timeouts)
        self._handle = ctypes.c_void_p(None)
        lib = _lib.load()
        size = ctypes.c_int64(0)
        nf, wt = _counter(nonfinite_count), _counter(wait_timeouts, "wait_timeouts")
        if config is None:
            name, model = "fsdp_clip_plan_create", (self.descs.array, self.descs.n)
            _check(lib.fsdp_clip_plan_workspace(*model, ctypes.byref(size)), "fsdp_clip_plan_workspace")
        else:
            cfg = config.to_c()
            name, model = "fsdp_clip_plan_create_ex", (self.descs.array_ex, self.descs.n, ctypes.byref(cfg))
            _check(lib.fsdp_clip_plan_workspace_ex(*model, ctypes.byref(size)), "fsdp_clip_plan_workspace_ex")
        if workspace is None or workspace.buf.numel() < size.value:
            workspace = Workspace(size.value, torch.device("cuda", torch.cuda.current_device()), zeroed=True)
        self.workspace = workspace
        _check(getattr(lib, name)(*model, int(gathers), workspace.buf.data_ptr(), workspace.buf.numel(), nf, wt,
                                  ctypes.byref(self._handle)), name)

    def launch(self, hparams, max_norm: float, norm: torch.Tensor,
               stream: Optional[torch.cuda.Stream] = None) -> None:
        """One step (hparams: AdamWHParams, or a StepConfig of the plan's
        optimizer); norm (fp32 CUDA scalar) receives the gradient's norm."""
        if not self._handle:
            raise RuntimeError("the model step was destroyed")
        s = self.workspace.on(stream)
        c = hparams.to_c()
        name = "fsdp_clip_plan_launch" if self.config is None else "fsdp_clip_plan_launch_ex"
        _check(getattr(_lib.load(), name)(self._handle, ctypes.byref(c), float(max_norm), _scalar(norm, "norm"),
                                          s.cuda_stream), name)

    def close(self) -> None:
        if self._handle:
            _check(_lib.load().fsdp_clip_plan_destroy(self._handle), "fsdp_clip_plan_destroy")
            self._handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
