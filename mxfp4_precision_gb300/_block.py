"""The operators between the GEMMs of a training step (RMS norm with the
residual's addition, SwiGLU, their gradients, gradient norm and clipping):
torch-tensor marshalling over include/mx.h, like _binding.py.

Matrices are 2-D CUDA tensors of torch.bfloat16 (or raw 16-bit patterns) or
torch.float32 whose rows are contiguous; a row pitch (a slice of columns) is
passed on.  Outputs and workspaces are allocated with torch unless given.  A
`stream` other than the current one becomes the current one for the call, so
that what is allocated belongs to it.
"""
from __future__ import annotations

from array import array
from operator import attrgetter
from typing import NamedTuple, Optional

import torch

from . import _binding as _b

FMT_MXFP4, FMT_MXFP8 = 1, 2
_BF16, _F32 = 0, 1
_TYPES = {torch.bfloat16: _BF16, torch.int16: _BF16, torch.uint16: _BF16, torch.float32: _F32}


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


def _stream(t: torch.Tensor) -> int:
    """The current stream of t's device, as torch's own launches look it up (torch.cuda.current_stream
    builds a Stream object first: 3 us of a call of 20)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _type(t: torch.Tensor, name: str) -> int:
    k = _TYPES.get(t.dtype)
    if k is None:
        raise ValueError(f"{name} must be bf16 (torch.bfloat16 or raw 16-bit patterns) or float32")
    return k


def _rows(t: torch.Tensor, name: str, shape=None):
    """(pointer, mx_type, pitch) of a matrix whose rows are contiguous."""
    kind = _TYPES.get(t.dtype)
    if kind is None:
        _type(t, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be 2-D" + (f" {tuple(shape)}" if shape else "") + f", got {tuple(t.shape)}")
    pitch, step = t.stride()
    rows, cols = t.shape
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), kind, pitch if rows > 1 else cols


def _vector(t: torch.Tensor, name: str, n: int):
    """(pointer, mx_type) of a contiguous vector of n elements."""
    kind = _TYPES.get(t.dtype)
    if kind is None:
        _type(t, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and [{n}], got {tuple(t.shape)}")
    return t.data_ptr(), kind


def _encoded(fmt, T: int, K: int, device):
    """Empty (codes, scales) of a row-direction encoding."""
    if fmt != FMT_MXFP8 and fmt != FMT_MXFP4:
        raise ValueError("fmt must be None, FMT_MXFP4 or FMT_MXFP8")
    # mx_scales_bytes(T, K), or one byte of an empty operand
    n = -(-T // 128) * 128 * (8 * -(-K // 256))
    return (torch.empty((T, K if fmt == FMT_MXFP8 else K // 2), dtype=torch.uint8, device=device),
            torch.empty(n or 1, dtype=torch.uint8, device=device))


def rmsnorm(x, weight, residual=None, eps: float = 1e-5, fmt=None, want_y: bool = True,
            out_h=None, stream=None) -> RMSNormOut:
    """h = x + residual, y = h * rstd * weight with rstd = 1 / sqrt(mean(h^2) + eps), over the
    rows of x [T, K]; y in bf16 (want_y) and / or encoded along its rows (fmt: FMT_MXFP4 or
    FMT_MXFP8) as the Fprop GEMM's operand.  h has the residual's type; out_h may be the residual
    itself.  See mx_rmsnorm."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm(x, weight, residual, eps, fmt, want_y, out_h)
    xp, xt, xs = _rows(x, "x")
    shape = x.shape
    T, K = shape
    d = x.device
    w, wt = _vector(weight, "weight", K)
    h, rp, rt, rs, hs = out_h, None, 0, 0, 0
    if residual is not None:
        rp, rt, rs = _rows(residual, "residual", shape)
        if h is None:
            h, hs = torch.empty(shape, dtype=residual.dtype, device=d), K
        else:
            _, ht, hs = _rows(h, "out_h", shape)
            if ht != rt:
                raise ValueError("out_h must have the residual's type")
    elif h is not None:
        raise ValueError("out_h needs a residual")
    y = torch.empty(shape, dtype=torch.bfloat16, device=d) if want_y else None
    codes, scales = _encoded(fmt, T, K, d) if fmt is not None else (None, None)
    rstd = torch.empty(T, dtype=torch.float32, device=d)
    st = (_b._lib or _b.lib()).mx_rmsnorm(
        xp, xt, xs, rp, rt, rs, w, wt, eps, T, K, None if h is None else h.data_ptr(), hs,
        None if y is None else y.data_ptr(), fmt or 0, None if codes is None else codes.data_ptr(),
        None if scales is None else scales.data_ptr(), rstd.data_ptr(), _stream(x))
    if st:
        _b._check(st, "mx_rmsnorm")
    return RMSNormOut(h, y, codes, scales, rstd)


def rmsnorm_backward_workspace_bytes(T: int, K: int) -> int:
    return int(_b.lib().mx_rmsnorm_backward_workspace_bytes(T, K))


def rmsnorm_backward(dy, h, weight, rstd, dres=None, want_dw: bool = True, ws=None, out_dx=None,
                     stream=None):
    """(dx, dw) of rmsnorm for y's gradient dy [T, K]: dx (of h's type) is the gradient of x and of
    the residual alike, dres (the stream's own gradient) added; dw fp32 [K].  out_dx may be dres
    itself.  See mx_rmsnorm_backward."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm_backward(dy, h, weight, rstd, dres, want_dw, ws, out_dx)
    dp, dt, ds = _rows(dy, "dy")
    shape = dy.shape
    T, K = shape
    d = dy.device
    hp, ht, hs = _rows(h, "h", shape)
    w, wt = _vector(weight, "weight", K)
    r, kind = _vector(rstd, "rstd", T)
    if kind != _F32:
        raise ValueError("rstd must be float32")
    gp, gs = None, 0
    if dres is not None:
        gp, gt, gs = _rows(dres, "dres", shape)
        if gt != ht:
            raise ValueError("dres must have h's type")
    if out_dx is None:
        out_dx = torch.empty(shape, dtype=h.dtype, device=d)
        op, os_ = out_dx.data_ptr(), K
    else:
        op, ot, os_ = _rows(out_dx, "out_dx", shape)
        if ot != ht:
            raise ValueError("out_dx must have h's type")
    L = _b._lib or _b.lib()
    dw, wp, n = None, None, 0
    if want_dw:
        dw = torch.empty(K, dtype=torch.float32, device=d)
        if ws is None:
            n = L.mx_rmsnorm_backward_workspace_bytes(T, K)
            ws = torch.empty(n or 1, dtype=torch.uint8, device=d)
        else:
            n = ws.numel() * ws.element_size()
        wp = _b._dev_ptr(ws, "workspace")
    st = L.mx_rmsnorm_backward(dp, dt, ds, hp, ht, hs, w, wt, r, gp, gs, T, K, op, os_,
                               None if dw is None else dw.data_ptr(), wp, n, _stream(dy))
    if st:
        _b._check(st, "mx_rmsnorm_backward")
    return out_dx, dw


def swiglu(gu, fmt=None, want_y: bool = True, stream=None) -> SwiGLUOut:
    """y = silu(g) * u of gu [T, 2F] = [g | u]: in bf16 (want_y) and / or encoded along its rows
    (fmt) as the down projection's Fprop operand.  See mx_swiglu."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return swiglu(gu, fmt, want_y)
    p, t, s = _rows(gu, "gu")
    T, F = gu.shape
    if F % 2:
        raise ValueError("gu must have an even number of columns")
    F //= 2
    d = gu.device
    y = torch.empty((T, F), dtype=torch.bfloat16, device=d) if want_y else None
    codes, scales = _encoded(fmt, T, F, d) if fmt is not None else (None, None)
    st = (_b._lib or _b.lib()).mx_swiglu(
        p, t, s, T, F, None if y is None else y.data_ptr(), fmt or 0,
        None if codes is None else codes.data_ptr(), None if scales is None else scales.data_ptr(),
        _stream(gu))
    if st:
        _b._check(st, "mx_swiglu")
    return SwiGLUOut(y, codes, scales)


def swiglu_backward(dy, gu, out=None, stream=None) -> torch.Tensor:
    """dgu [T, 2F] in bf16 for y's gradient dy [T, F].  See mx_swiglu_backward."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return swiglu_backward(dy, gu, out)
    dp, dt, ds = _rows(dy, "dy")
    T, F = dy.shape
    gp, gt, gs = _rows(gu, "gu", (T, 2 * F))
    if out is None:
        out = torch.empty((T, 2 * F), dtype=torch.bfloat16, device=dy.device)
    elif tuple(out.shape) != (T, 2 * F) or _type(out, "out") != _BF16:
        raise ValueError(f"out must be bf16 [{T}, {2 * F}]")
    st = (_b._lib or _b.lib()).mx_swiglu_backward(dp, dt, ds, gp, gt, gs, T, F, _b._dev_ptr(out, "out"),
                                                  _stream(dy))
    if st:
        _b._check(st, "mx_swiglu_backward")
    return out


def grad_workspace_bytes(count: int) -> int:
    return int(_b.lib().mx_grad_workspace_bytes(count))


_DATA_PTR, _NUMEL, _IS_CONTIGUOUS = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous
_IS_CUDA, _DTYPE = attrgetter("is_cuda"), attrgetter("dtype")


def _tables(tensors, name: str):
    """Host arrays (pointers, sizes, types) of contiguous CUDA tensors: one pass of `map` for each, a
    third of the time of a loop over the tensors."""
    if not all(map(_IS_CUDA, tensors)):
        raise ValueError(f"{name} must be a CUDA tensor")
    if not all(map(_IS_CONTIGUOUS, tensors)):
        raise ValueError(f"{name} must be contiguous")
    try:
        types = array("i", map(_TYPES.__getitem__, map(_DTYPE, tensors)))
    except KeyError:
        raise ValueError(f"{name} must be bf16 (torch.bfloat16 or raw 16-bit patterns) or float32") from None
    return array("Q", map(_DATA_PTR, tensors)), array("q", map(_NUMEL, tensors)), types


def _at(a):
    return None if a is None else a.buffer_info()[0]


def _grad_buffers(tensors, ws):
    d = tensors[0].device if tensors else "cuda"
    norm = torch.empty(1, dtype=torch.float32, device=d)
    if ws is None:
        ws = torch.empty(grad_workspace_bytes(len(tensors)) or 1, dtype=torch.uint8, device=d)
    return norm, ws


def grad_norm(tensors, ws=None, stream=None) -> torch.Tensor:
    """L2 norm over all elements of a list of contiguous bf16 / fp32 CUDA tensors, as a
    one-element fp32 device tensor.  See mx_grad_norm."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return grad_norm(tensors, ws)
    tensors = list(tensors)
    p, n, t = _tables(tensors, "gradient")
    norm, ws = _grad_buffers(tensors, ws)
    st = _b.lib().mx_grad_norm(_at(p), _at(n), _at(t), len(tensors), norm.data_ptr(), ws.data_ptr(), ws.numel(),
                               _stream(norm))
    _b._check(st, "mx_grad_norm")
    return norm


def clip_grads(tensors, max_norm: float, out=None, eps: float = 1e-6, ws=None,
               stream=None) -> torch.Tensor:
    """Scales every gradient by min(1, max_norm / (norm + eps)), norm over all of them: in place, or
    into the tensors of `out` (same sizes, bf16 or fp32).  Returns the norm before clipping, a
    one-element fp32 device tensor.  See mx_clip_grads."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return clip_grads(tensors, max_norm, out, eps, ws)
    tensors = list(tensors)
    p, n, t = _tables(tensors, "gradient")
    op = ot = None
    if out is not None:
        out = list(out)
        op, on, ot = _tables(out, "out")
        if on != n:
            raise ValueError("out must hold one tensor of the same size for each gradient")
    norm, ws = _grad_buffers(tensors, ws)
    st = _b.lib().mx_clip_grads(_at(p), _at(n), _at(t), _at(op), _at(ot), len(tensors), max_norm, eps, norm.data_ptr(),
                                ws.data_ptr(), ws.numel(), _stream(norm))
    _b._check(st, "mx_clip_grads")
    return norm
