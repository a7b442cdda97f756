"""The operators between the GEMMs of a training step (RMS norm with the
residual's addition, SwiGLU, their gradients, gradient norm and clipping).

Matrices are 2-D CUDA tensors of torch.bfloat16 (or raw 16-bit patterns) or
torch.float32 whose rows are contiguous; a row pitch (a slice of columns) is
passed on.  All tensors of a call are on one device.  Outputs and workspaces are
allocated with torch unless given.  A `stream` other than the current one (of the
tensors' device) becomes the current one for the call, so that what is allocated
belongs to it.  None of them records an autograd node: the gradients are calls of
their own.

The tensors are checked and unpacked in ``_build/mx_torch.so``
(csrc/mx_torch.cpp), which calls the C ABI in include/mx.h; ValueError for
tensors it does not take, MXError for a status.
"""
from __future__ import annotations

import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from . import _binding as _b
from .build import TORCH_LIB, fits_torch

FMT_MXFP4, FMT_MXFP8 = 1, 2

_calls = None


def _load():
    """The module of the entry points; raises if it has not been built."""
    global _calls
    with _b._lock:
        if _calls is None:
            if not os.path.exists(TORCH_LIB):
                raise RuntimeError(
                    f"MXFP4 torch entry points not found at {TORCH_LIB}; build them with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            if not fits_torch():
                raise RuntimeError(
                    f"{TORCH_LIB} was built against another torch or Python; build it again with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            spec = importlib.util.spec_from_file_location("mx_torch", TORCH_LIB)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.set_check(_b._check)
            _calls = module
    return _calls


def _on(stream, tensor):
    """`stream` as the current one; a stream of another device would leave the call on its device's own."""
    if getattr(tensor, "is_cuda", False) and tensor.device != stream.device:
        raise ValueError(f"stream must be on {tensor.device} like the call's tensors, not on {stream.device}")
    return torch.cuda.stream(stream)


class RMSNormOut(NamedTuple):
    """h: the new stream (None without a residual); y: bf16 (None if not wanted);
    codes, scales: the encoded y (None without fmt); rstd: fp32 [T]."""
    h: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]
    rstd: torch.Tensor


class SwiGLUOut(NamedTuple):
    y: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def rmsnorm(x, weight, residual=None, eps: float = 1e-5, fmt=None, want_y: bool = True,
            out_h=None, stream=None) -> RMSNormOut:
    """h = x + residual, y = h * rstd * weight with rstd = 1 / sqrt(mean(h^2) + eps), over the
    rows of x [T, K]; y in bf16 (want_y) and / or encoded along its rows (fmt: FMT_MXFP4 or
    FMT_MXFP8) as the Fprop GEMM's operand.  h has the residual's type; out_h may be the residual
    itself.  See mx_rmsnorm."""
    if stream is not None:
        with _on(stream, x):
            return rmsnorm(x, weight, residual, eps, fmt, want_y, out_h)
    return RMSNormOut._make((_calls or _load()).rmsnorm(x, weight, residual, eps, fmt, want_y, out_h))


def rmsnorm_backward_workspace_bytes(T: int, K: int) -> int:
    return int(_b.lib().mx_rmsnorm_backward_workspace_bytes(T, K))


def rmsnorm_backward(dy, h, weight, rstd, dres=None, want_dw: bool = True, ws=None, out_dx=None,
                     stream=None):
    """(dx, dw) of rmsnorm for y's gradient dy [T, K]: dx (of h's type) is the gradient of x and of
    the residual alike, dres (the stream's own gradient) added; dw fp32 [K].  out_dx may be dres
    itself.  See mx_rmsnorm_backward."""
    if stream is not None:
        with _on(stream, dy):
            return rmsnorm_backward(dy, h, weight, rstd, dres, want_dw, ws, out_dx)
    return (_calls or _load()).rmsnorm_backward(dy, h, weight, rstd, dres, want_dw, ws, out_dx)


def swiglu(gu, fmt=None, want_y: bool = True, stream=None) -> SwiGLUOut:
    """y = silu(g) * u of gu [T, 2F] = [g | u]: in bf16 (want_y) and / or encoded along its rows
    (fmt) as the down projection's Fprop operand.  See mx_swiglu."""
    if stream is not None:
        with _on(stream, gu):
            return swiglu(gu, fmt, want_y)
    return SwiGLUOut._make((_calls or _load()).swiglu(gu, fmt, want_y))


def swiglu_backward(dy, gu, out=None, stream=None) -> torch.Tensor:
    """dgu [T, 2F] in bf16 for y's gradient dy [T, F].  See mx_swiglu_backward."""
    if stream is not None:
        with _on(stream, dy):
            return swiglu_backward(dy, gu, out)
    return (_calls or _load()).swiglu_backward(dy, gu, out)


def grad_workspace_bytes(count: int) -> int:
    return int(_b.lib().mx_grad_workspace_bytes(count))


def grad_norm(tensors, ws=None, stream=None) -> torch.Tensor:
    """L2 norm over all elements of a list of contiguous bf16 / fp32 CUDA tensors, as a
    one-element fp32 device tensor.  See mx_grad_norm."""
    tensors = list(tensors)
    if stream is not None:
        with _on(stream, tensors[0] if tensors else None):
            return grad_norm(tensors, ws)
    if not tensors:
        return torch.zeros(1, dtype=torch.float32, device="cuda")
    return (_calls or _load()).clip(tensors, None, False, 0.0, 0.0, ws)


def clip_grads(tensors, max_norm: float, out=None, eps: float = 1e-6, ws=None,
               stream=None) -> torch.Tensor:
    """Scales every gradient by min(1, max_norm / (norm + eps)), norm over all of them: in place, or
    into the tensors of `out` (same sizes, bf16 or fp32).  Returns the norm before clipping, a
    one-element fp32 device tensor.  See mx_clip_grads."""
    tensors = list(tensors)
    if stream is not None:
        with _on(stream, tensors[0] if tensors else None):
            return clip_grads(tensors, max_norm, out, eps, ws)
    if not tensors:
        return torch.zeros(1, dtype=torch.float32, device="cuda")
    return (_calls or _load()).clip(tensors, None if out is None else list(out), True, max_norm, eps, ws)
