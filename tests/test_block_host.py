"""Host-only checks of the operators between the GEMMs: every bad argument is
refused with its documented status before anything is launched, empty calls
return at once, workspaces have their documented sizes.  No call here reaches
a GPU."""
import ctypes

import pytest

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build as mxbuild

OK, ARG, SHAPE, ALIGN, WS, UNSUP = 0, 1, 2, 3, 4, 7
A = [0x10000 * (i + 1) for i in range(12)]     # distinct aligned addresses, never read


@pytest.fixture(scope="module")
def L():
    mxbuild.build()
    return mx.lib()


def _norm(L, x=A[0], xt=1, xp=512, res=A[1], rt=0, rp=512, w=A[2], wt=0, eps=1e-5, T=4, K=512, h=A[3],
          hp=512, y=A[4], fmt=2, codes=A[5], scales=A[6], rstd=A[7]):
    return L.mx_rmsnorm(x, xt, xp, res, rt, rp, w, wt, eps, T, K, h, hp, y, fmt, codes, scales, rstd, None)


def test_norm_refusals(L):
    for bad in (dict(xt=2), dict(rt=-1), dict(wt=7), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None),
                dict(w=None), dict(fmt=3), dict(fmt=0), dict(codes=None), dict(scales=None),
                dict(res=None)):
        assert _norm(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(K=-8), dict(T=1 << 31), dict(xp=504), dict(rp=256), dict(hp=8),
                dict(K=488, xp=512)):
        assert _norm(L, **bad) == SHAPE, bad
    for bad in (dict(x=A[0] + 2), dict(res=A[1] + 8), dict(w=A[2] + 2), dict(h=A[3] + 4), dict(y=A[4] + 2),
                dict(codes=A[5] + 8), dict(scales=A[6] + 4), dict(rstd=A[7] + 4), dict(xp=516), dict(rp=513),
                dict(hp=515), dict(K=510, fmt=0, codes=None, scales=None)):
        assert _norm(L, **bad) == ALIGN, bad
    assert _norm(L, K=40000 // 32 * 32, xp=40000, rp=40000, hp=40000) == UNSUP
    assert _norm(L, T=0) == OK and _norm(L, K=0) == OK
    assert _norm(L, T=0, codes=None, scales=None, x=None) == OK


def _norm_b(L, dy=A[0], dt=1, dp=512, h=A[1], ht=0, hp=512, w=A[2], wt=0, rstd=A[3], dres=A[4], gp=512, T=4,
            K=512, dx=A[5], xp=512, dw=A[6], ws=A[7], n=1 << 30):
    return L.mx_rmsnorm_backward(dy, dt, dp, h, ht, hp, w, wt, rstd, dres, gp, T, K, dx, xp, dw, ws, n, None)


def test_norm_backward_refusals(L):
    for bad in (dict(dt=2), dict(ht=5), dict(wt=-1), dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None),
                dict(dx=None)):
        assert _norm_b(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(K=-8), dict(dp=504), dict(hp=0), dict(gp=8), dict(xp=16)):
        assert _norm_b(L, **bad) == SHAPE, bad
    for bad in (dict(dy=A[0] + 4), dict(h=A[1] + 2), dict(dres=A[4] + 2), dict(dx=A[5] + 8), dict(dw=A[6] + 4),
                dict(w=A[2] + 2), dict(rstd=A[3] + 4), dict(ws=A[7] + 16), dict(dp=514), dict(K=508)):
        assert _norm_b(L, **bad) == ALIGN, bad
    assert _norm_b(L, ws=None) == WS and _norm_b(L, n=16) == WS
    assert _norm_b(L, K=32776, dp=32776, hp=32776, gp=32776, xp=32776) == UNSUP
    assert _norm_b(L, K=0) == OK and _norm_b(L, T=0, dw=None) == OK
    assert mx.rmsnorm_backward_workspace_bytes(0, 512) == 0
    assert mx.rmsnorm_backward_workspace_bytes(4, 0) == 0
    for T, K in ((1, 8), (97, 2080), (8192, 4096), (1 << 20, 32768)):
        n = mx.rmsnorm_backward_workspace_bytes(T, K)
        assert n % 256 == 0 and 4 * K <= n <= 1 << 28


def _glu(L, gu=A[0], t=1, p=1024, T=4, F=512, y=A[1], fmt=1, codes=A[2], scales=A[3]):
    return L.mx_swiglu(gu, t, p, T, F, y, fmt, codes, scales, None)


def _glu_b(L, dy=A[0], dt=1, dp=512, gu=A[1], t=0, p=1024, T=4, F=512, out=A[2]):
    return L.mx_swiglu_backward(dy, dt, dp, gu, t, p, T, F, out, None)


def test_swiglu_refusals(L):
    for bad in (dict(t=2), dict(gu=None), dict(fmt=-1), dict(codes=None), dict(fmt=0)):
        assert _glu(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(F=-1), dict(p=1016), dict(F=488)):
        assert _glu(L, **bad) == SHAPE, bad
    for bad in (dict(gu=A[0] + 8), dict(y=A[1] + 2), dict(codes=A[2] + 1), dict(p=1026),
                dict(F=508, fmt=0, codes=None, scales=None)):
        assert _glu(L, **bad) == ALIGN, bad
    assert _glu(L, T=0) == OK and _glu(L, F=0) == OK
    for bad in (dict(dt=2), dict(t=2), dict(dy=None), dict(gu=None), dict(out=None)):
        assert _glu_b(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(dp=504), dict(p=1000)):
        assert _glu_b(L, **bad) == SHAPE, bad
    for bad in (dict(dy=A[0] + 4), dict(out=A[2] + 8), dict(dp=516), dict(F=508)):
        assert _glu_b(L, **bad) == ALIGN, bad
    assert _glu_b(L, T=0) == OK and _glu_b(L, F=0) == OK


def _clip(L, ptrs=(A[0], A[1]), sizes=(100, 7), types=(1, 0), outs=(A[2], A[3]), out_types=(0, 0), count=2,
          max_norm=1.0, eps=1e-6, norm=A[4], ws=A[5], n=1 << 20, only_norm=False):
    arr = lambda t, v: None if v is None else (t * len(v))(*v)  # noqa: E731
    p, s, t = arr(ctypes.c_void_p, ptrs), arr(ctypes.c_int64, sizes), arr(ctypes.c_int, types)
    if only_norm:
        return L.mx_grad_norm(p, s, t, count, norm, ws, n, None)
    return L.mx_clip_grads(p, s, t, arr(ctypes.c_void_p, outs), arr(ctypes.c_int, out_types), count, max_norm,
                           eps, norm, ws, n, None)


def test_clip_refusals(L):
    for bad in (dict(ptrs=None), dict(sizes=None), dict(types=None), dict(out_types=None), dict(types=(1, 2)),
                dict(out_types=(3, 0)), dict(ptrs=(A[0], None)), dict(outs=(None, A[3])), dict(norm=None),
                dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(eps=float("nan")),
                dict(outs=(A[0], A[3]))):                     # in place with another type
        assert _clip(L, **bad) == ARG, bad
    for bad in (dict(sizes=(100, -1)), dict(count=-1), dict(count=(1 << 20) + 1)):
        assert _clip(L, **bad) == SHAPE, bad
    for bad in (dict(ptrs=(A[0] + 2, A[1])), dict(ptrs=(A[0], A[1] + 1)), dict(outs=(A[2] + 1, A[3])),
                dict(norm=A[4] + 2), dict(ws=A[5] + 8)):
        assert _clip(L, **bad) == ALIGN, bad
    assert _clip(L, ws=None) == WS and _clip(L, n=8) == WS
    assert _clip(L, only_norm=True, ws=None) == WS and _clip(L, only_norm=True, norm=None) == ARG
    assert mx.grad_workspace_bytes(0) == 0 and mx.grad_workspace_bytes(1) % 256 == 0
    assert mx.grad_workspace_bytes(5000) >= mx.grad_workspace_bytes(1)


def test_python_refusals():
    import torch
    x = torch.zeros(4, 64)
    for call in (lambda: mx.rmsnorm(x, x[0]), lambda: mx.swiglu(x), lambda: mx.swiglu_backward(x, x),
                 lambda: mx.rmsnorm_backward(x, x, x[0], x[:, 0]), lambda: mx.grad_norm([x]),
                 lambda: mx.clip_grads([x], 1.0)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
