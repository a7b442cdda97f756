"""Host-only checks of the products with an epilogue and by expert: every bad
argument is refused with its documented status before anything is launched,
empty calls return at once, workspaces and row counts are as documented.  No call
here reaches a GPU."""
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build as mxbuild
from tests.test_block_devices import Placed

OK, ARG, SHAPE, ALIGN, WS, UNSUP = 0, 1, 2, 3, 4, 7
A = [0x10000 * (i + 1) for i in range(16)]     # distinct aligned addresses, never read


@pytest.fixture(scope="module")
def L():
    mxbuild.build()
    return mx.lib()


def _gemm(L, aq=A[0], as_=A[1], bq=A[2], bs=A[3], fmt=1, M=4, N=512, K=64, bias=A[4], bt=0, act=3, res=A[5], rt=1, rp=512, y=A[6], yt=0,
          z=A[7], ef=2, codes=A[8], scales=A[9]):
    return L.mx_gemm_bias_act(aq, as_, bq, bs, fmt, M, N, K, bias, bt, act, res, rt, rp, y, yt, z, ef, codes, scales, None)


def test_gemm_refusals(L):
    for bad in (dict(fmt=0), dict(fmt=3), dict(bt=2), dict(act=6), dict(act=-1), dict(rt=5), dict(yt=-1), dict(ef=3), dict(codes=None),
                dict(ef=0), dict(aq=None), dict(as_=None), dict(bq=None), dict(bs=None),
                dict(y=None, z=None, ef=0, codes=None, scales=None)):
        assert _gemm(L, **bad) == ARG, bad
    for bad in (dict(M=-1), dict(N=-8), dict(K=-32), dict(K=48), dict(M=1 << 31), dict(N=488, rp=512), dict(rp=504)):
        assert _gemm(L, **bad) == SHAPE, bad
    for bad in (dict(N=508, rp=512, ef=0, codes=None, scales=None), dict(aq=A[0] + 8), dict(as_=A[1] + 4), dict(bq=A[2] + 1), dict(bs=A[3] + 8),
                dict(bias=A[4] + 2), dict(res=A[5] + 4), dict(rp=516), dict(y=A[6] + 8), dict(z=A[7] + 2), dict(codes=A[8] + 8),
                dict(scales=A[9] + 4)):
        assert _gemm(L, **bad) == ALIGN, bad
    assert _gemm(L, M=0) == OK and _gemm(L, N=0) == OK
    assert _gemm(L, M=0, aq=None, y=None, z=None, ef=0, codes=None, scales=None) == OK


def _back(L, dy=A[0], dt=1, dp=512, z=A[1], zt=0, zp=512, act=5, T=4, N=512, dz=A[2], ef=1, codes=A[3], scales=A[4], db=A[5], ws=A[6],
          n=1 << 30):
    return L.mx_bias_act_backward(dy, dt, dp, z, zt, zp, act, T, N, dz, ef, codes, scales, db, ws, n, None)


def test_backward_refusals(L):
    for bad in (dict(dt=2), dict(zt=3), dict(act=7), dict(dy=None), dict(z=None), dict(ef=4), dict(codes=None),
                dict(dz=None, ef=0, codes=None, scales=None, db=None)):
        assert _back(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(N=-1), dict(dp=8), dict(zp=504), dict(N=488)):
        assert _back(L, **bad) == SHAPE, bad
    for bad in (dict(dy=A[0] + 4), dict(z=A[1] + 2), dict(dz=A[2] + 8), dict(db=A[5] + 4), dict(dp=514), dict(zp=515),
                dict(T=4000, ws=A[6] + 16)):
        assert _back(L, **bad) == ALIGN, bad
    assert _back(L, T=4000, ws=None) == WS and _back(L, T=4000, n=256) == WS
    assert _back(L, N=0) == OK and _back(L, T=0, db=None) == OK
    assert mx.bias_act_backward_workspace_bytes(97, 2080) == 0 == mx.bias_act_backward_workspace_bytes(0, 64)
    for T, N in ((129, 8), (8192, 14336), (1 << 20, 32768)):
        n = mx.bias_act_backward_workspace_bytes(T, N)
        assert n % 256 == 0 and 8 * N <= n <= 128 * 4 * N + 256


def test_rows_that_the_segments_can_take():
    assert mx.expert_rows(0, 2, 4) == 0 == mx.expert_rows(4, 0, 4)
    assert mx.expert_rows(1, 1, 1) == 128 and mx.expert_rows(1, 1, 64) == 128
    assert mx.expert_rows(2, 1, 64) == 256 and mx.expert_rows(129, 1, 1) == 256
    for T, picks, E in ((9, 4, 16), (8192, 2, 8), (301, 2, 16)):
        n = T * picks
        # the fullest way to cut n rows into segments of 128
        most = n if E == 0 else 128 * min(E - 1, n - 1) + -(-(n - min(E - 1, n - 1)) // 128) * 128
        assert most <= mx.expert_rows(T, picks, E) <= n + 127 * E and mx.expert_rows(T, picks, E) % 128 == 0


def _plan(L, ix=A[0], b=4, T=9, k=2, E=8, off=A[1], cnt=A[2], slot=A[3], src=A[4], ws=A[5], n=1 << 30):
    return L.mx_expert_plan(ix, b, T, k, E, off, cnt, slot, src, ws, n, None)


def test_plan_refusals(L):
    for bad in (dict(b=2), dict(ix=None), dict(off=None), dict(cnt=None), dict(slot=None), dict(src=None)):
        assert _plan(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(k=-1), dict(E=0), dict(E=-3), dict(T=1 << 30, k=4), dict(T=(1 << 31) - 100, k=1)):
        assert _plan(L, **bad) == SHAPE, bad
    for bad in (dict(ix=A[0] + 2), dict(b=8, ix=A[0] + 4), dict(off=A[1] + 4), dict(cnt=A[2] + 8), dict(slot=A[3] + 4), dict(src=A[4] + 4),
                dict(T=5000, ws=A[5] + 16)):
        assert _plan(L, **bad) == ALIGN, bad
    assert _plan(L, E=513) == UNSUP
    assert _plan(L, T=5000, ws=None) == WS and _plan(L, T=5000, n=0) == WS
    assert mx.expert_plan_workspace_bytes(9, 2, 8) == 0 and mx.expert_plan_workspace_bytes(5000, 2, 8) % 256 == 0


def _in(L, x=A[0], t=0, p=512, slot=A[1], src=A[2], T=4, k=2, P=256, K=512, y=A[3], ef=1, codes=A[4], scales=A[5]):
    return L.mx_expert_dispatch(x, t, p, slot, src, T, k, P, K, y, ef, codes, scales, None)


def _out(L, r=A[0], t=0, p=512, slot=A[1], w=A[2], T=4, k=2, P=256, K=512, res=A[3], rt=0, rp=512, y=A[4], yt=0):
    return L.mx_expert_combine(r, t, p, slot, w, T, k, P, K, res, rt, rp, y, yt, None)


def _grad(L, dy=A[0], dt=0, dp=512, r=A[1], rt=0, rp=512, slot=A[2], src=A[3], w=A[4], T=4, k=2, P=256, K=512, dr=A[5], ef=2, codes=A[6],
          scales=A[7], dw=A[8]):
    return L.mx_expert_combine_backward(dy, dt, dp, r, rt, rp, slot, src, w, T, k, P, K, dr, ef, codes, scales, dw, None)


def test_rows_refusals(L):
    for bad in (dict(x=None), dict(t=2), dict(slot=None), dict(src=None), dict(ef=3), dict(codes=None),
                dict(y=None, ef=0, codes=None, scales=None)):
        assert _in(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(P=100), dict(P=-128), dict(K=-8), dict(p=8), dict(K=488)):
        assert _in(L, **bad) == SHAPE, bad
    for bad in (dict(x=A[0] + 2), dict(slot=A[1] + 4), dict(src=A[2] + 8), dict(y=A[3] + 2), dict(codes=A[4] + 8), dict(p=516),
                dict(K=508, ef=0, codes=None, scales=None)):
        assert _in(L, **bad) == ALIGN, bad
    assert _in(L, P=0) == OK and _in(L, K=0) == OK
    for bad in (dict(r=None), dict(t=-1), dict(slot=None), dict(rt=9), dict(y=None), dict(yt=3)):
        assert _out(L, **bad) == ARG, bad
    for bad in (dict(T=-1), dict(P=130), dict(p=504), dict(rp=8)):
        assert _out(L, **bad) == SHAPE, bad
    for bad in (dict(r=A[0] + 2), dict(slot=A[1] + 4), dict(w=A[2] + 4), dict(res=A[3] + 8), dict(y=A[4] + 8), dict(K=500, p=504, rp=504)):
        assert _out(L, **bad) == ALIGN, bad
    assert _out(L, T=0) == OK and _out(L, K=0) == OK
    for bad in (dict(dy=None), dict(dt=2), dict(rt=2), dict(r=None), dict(slot=None), dict(src=None), dict(w=None), dict(codes=None),
                dict(dr=None, ef=0, codes=None, scales=None, dw=None)):
        assert _grad(L, **bad) == ARG, bad
    for bad in (dict(P=64), dict(T=-2), dict(dp=8), dict(rp=256), dict(K=488)):
        assert _grad(L, **bad) == SHAPE, bad
    for bad in (dict(dy=A[0] + 4), dict(r=A[1] + 2), dict(slot=A[2] + 4), dict(src=A[3] + 4), dict(w=A[4] + 8), dict(dr=A[5] + 2),
                dict(dw=A[8] + 4), dict(dp=514), dict(rp=518)):
        assert _grad(L, **bad) == ALIGN, bad
    assert _grad(L, K=0, T=0) == OK and _grad(L, T=0, dr=None, ef=0, codes=None, scales=None) == OK


def _rows(L, aq=A[0], as_=A[1], bq=A[2], bs=A[3], fmt=2, off=A[4], cnt=A[5], E=4, P=512, N=256, K=64, bias=A[6], bt=1, act=1, y=A[7], yt=1,
          z=A[8], ef=1, codes=A[9], scales=A[10]):
    return L.mx_gemm_experts(aq, as_, bq, bs, fmt, off, cnt, E, P, N, K, bias, bt, act, y, yt, z, ef, codes, scales, None)


def _depth(L, aq=A[0], as_=A[1], bq=A[2], bs=A[3], fmt=1, off=A[4], E=4, P=512, M=256, N=64, c=A[5], ct=1):
    return L.mx_gemm_experts_wgrad(aq, as_, bq, bs, fmt, off, E, P, M, N, c, ct, None)


def _linear(L, dy=A[0], x=A[1], fmt=1, off=A[2], E=4, P=512, N=256, K=64, rot=1, nb=32, rnd=0, dw=A[3], dt=1, ws=A[4], n=1 << 30):
    return L.mx_linear_experts_wgrad(dy, x, fmt, off, E, P, N, K, rot, nb, rnd, 0, dw, dt, ws, n, None)


def test_experts_refusals(L):
    for bad in (dict(fmt=0), dict(off=None), dict(cnt=None), dict(aq=None), dict(bs=None), dict(bt=2), dict(act=9), dict(yt=2), dict(codes=None),
                dict(y=None, z=None, ef=0, codes=None, scales=None)):
        assert _rows(L, **bad) == ARG, bad
    for bad in (dict(E=0), dict(P=500), dict(P=-128), dict(N=-8), dict(K=40), dict(E=512, N=1 << 23), dict(N=264)):
        assert _rows(L, **bad) == SHAPE, bad
    for bad in (dict(off=A[4] + 4), dict(cnt=A[5] + 4), dict(N=252, ef=0, codes=None, scales=None), dict(y=A[7] + 8), dict(bias=A[6] + 4)):
        assert _rows(L, **bad) == ALIGN, bad
    assert _rows(L, E=513) == UNSUP
    assert _rows(L, P=0) == OK and _rows(L, N=0) == OK
    for bad in (dict(fmt=4), dict(off=None), dict(c=None), dict(aq=None), dict(ct=2)):
        assert _depth(L, **bad) == ARG, bad
    for bad in (dict(E=0), dict(P=96), dict(M=-1), dict(N=-1)):
        assert _depth(L, **bad) == SHAPE, bad
    for bad in (dict(N=60), dict(c=A[5] + 4), dict(off=A[4] + 8), dict(aq=A[0] + 8)):
        assert _depth(L, **bad) == ALIGN, bad
    assert _depth(L, E=1000) == UNSUP and _depth(L, M=0) == OK and _depth(L, N=0) == OK
    for bad in (dict(fmt=0), dict(off=None), dict(dy=None), dict(x=None), dict(dw=None), dict(rot=3), dict(nb=48), dict(rnd=2), dict(dt=4)):
        assert _linear(L, **bad) == ARG, bad
    for bad in (dict(P=100), dict(E=0), dict(N=-8)):
        assert _linear(L, **bad) == SHAPE, bad
    for bad in (dict(N=252), dict(K=60), dict(dy=A[0] + 2), dict(dw=A[3] + 4), dict(ws=A[4] + 64)):
        assert _linear(L, **bad) == ALIGN, bad
    for bad in (dict(nb=256), dict(fmt=2), dict(fmt=2, rot=0, rnd=1), dict(E=513)):
        assert _linear(L, **bad) == UNSUP, bad
    assert _linear(L, ws=None) == WS and _linear(L, n=1000) == WS and _linear(L, N=0) == OK
    n = mx.linear_experts_wgrad_workspace_bytes(mx.FMT_MXFP4, 512, 256, 64)
    assert n == mx.linear_workspace_bytes(mx.OP_WGRAD, 512, 256, 64) - 256  # that one also holds counters
    assert mx.linear_experts_wgrad_workspace_bytes(mx.FMT_MXFP8, 512, 256, 64) == mx.linear_wgrad_mxfp8_workspace_bytes(512, 256, 64)


def test_quantize_refusals(L):
    q = lambda src=A[0], E=3, rows=64, cols=96, fmt=1, c=1, rot=0, nb=32, codes=A[1], scales=A[2]: (  # noqa: E731
        L.mx_quantize_experts(src, E, rows, cols, fmt, c, rot, nb, 0, codes, scales, None))
    assert q(fmt=0) == ARG and q(c=2) == ARG and q(src=None) == ARG and q(rot=4) == ARG
    assert q(E=-1) == SHAPE and q(cols=40) == SHAPE and q(rot=1, nb=64) == SHAPE
    assert q(rows=64, cols=100, c=0) == ALIGN and q(codes=A[1] + 8) == ALIGN
    assert q(fmt=2) == UNSUP and q(fmt=2, c=0, rot=1) == UNSUP and q(E=513) == UNSUP
    assert q(E=0) == OK and q(rows=0) == OK


# ---------------------------------------------------------------------------- from torch
F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
T, PICKS, E, P, N, K = 8, 2, 4, 512, 64, 96


def _at(shape, dtype=F32, device="cuda:0"):
    return Placed(shape, dtype, device)


def _operands(a, b):
    return [((a, K // 2), U8), ((mx.scales_bytes(a, K),), U8), ((b, K // 2), U8), ((mx.scales_bytes(b, K),), U8)]


PLAN = [((E + 1,), I32), ((E,), I32), ((T, PICKS), I32), ((P,), I32)]


def _calls():
    """(call on a list of tensors, their shapes and types)"""
    plan = lambda t: mx.ExpertPlan(*t)  # noqa: E731
    experts = [((P, K // 2), U8), ((mx.scales_bytes(P, K),), U8), ((E * N, K // 2), U8), ((E * mx.scales_bytes(N, K),), U8)]
    depth = [((N, P // 2), U8), ((mx.scales_bytes(N, P),), U8), ((K, P // 2), U8), ((mx.scales_bytes(K, P),), U8)]
    return {
        "gemm_bias_act": (lambda t: mx.gemm_bias_act(*t[:4], T, N, K, bias=t[4], residual=t[5], out=t[6]),
                          _operands(T, N) + [((N,), F32), ((T, N), F32), ((T, N), F32)]),
        "bias_act_backward": (lambda t: mx.bias_act_backward(t[0], t[1], mx.ACT_RELU, ws=t[2]), [((T, N), F32), ((T, N), BF16), ((256,), U8)]),
        "expert_plan": (lambda t: mx.expert_plan(t[0], E, ws=t[1]), [((T, PICKS), I32), ((256,), U8)]),
        "expert_dispatch": (lambda t: mx.expert_dispatch(t[0], plan(t[1:5])), [((T, K), F32)] + PLAN),
        "expert_combine": (lambda t: mx.expert_combine(t[0], plan(t[1:5]), t[5], t[6], out=t[7]),
                           [((P, K), F32)] + PLAN + [((T, PICKS), F32), ((T, K), F32), ((T, K), F32)]),
        "expert_combine_backward": (lambda t: mx.expert_combine_backward(t[0], t[1], plan(t[2:6]), t[6]),
                                    [((T, K), F32), ((P, K), F32)] + PLAN + [((T, PICKS), F32)]),
        "gemm_experts": (lambda t: mx.gemm_experts(*t[:4], plan(t[4:8]), N, K, bias=t[8]), experts + PLAN + [((E, N), F32)]),
        "gemm_experts_wgrad": (lambda t: mx.gemm_experts_wgrad(*t[:4], plan(t[4:8]), N, K, out=t[8]), depth + PLAN + [((E, N, K), F32)]),
        "linear_experts_wgrad": (lambda t: mx.linear_experts_wgrad(t[0], t[1], plan(t[2:6]), ws=t[6], out=t[7]),
                                 [((P, N), BF16), ((P, K), BF16)] + PLAN + [((1 << 20,), U8), ((E, N, K), F32)]),
    }


NAMES = ["gemm_bias_act", "bias_act_backward", "expert_plan", "expert_dispatch", "expert_combine", "expert_combine_backward", "gemm_experts",
         "gemm_experts_wgrad", "linear_experts_wgrad"]


@pytest.mark.parametrize("name", NAMES)
def test_one_tensor_elsewhere_is_refused(L, name):
    call, shapes = _calls()[name]
    for where in range(1, len(shapes)):
        with pytest.raises(ValueError, match="must be on cuda:[01] like"):
            call([_at(s, t, "cuda:1" if i == where else "cuda:0") for i, (s, t) in enumerate(shapes)])


def test_a_stream_of_another_device_is_refused(L):
    from types import SimpleNamespace
    stream = SimpleNamespace(device=torch.device("cuda:1"))
    x, plan = _at((P, K)), mx.ExpertPlan(*(_at(s, t) for s, t in PLAN))
    codes = _at((P, K // 2), U8)
    for call in (lambda: mx.gemm_bias_act(codes, codes, codes, codes, P, N, K, stream=stream), lambda: mx.bias_act_backward(x, stream=stream),
                 lambda: mx.expert_plan(x, E, stream=stream), lambda: mx.expert_dispatch(x, plan, stream=stream),
                 lambda: mx.expert_combine(x, plan, stream=stream), lambda: mx.expert_combine_backward(x, x, plan, x, stream=stream),
                 lambda: mx.quantize_experts(x, stream=stream), lambda: mx.gemm_experts(codes, codes, codes, codes, plan, N, K, stream=stream),
                 lambda: mx.gemm_experts_wgrad(codes, codes, codes, codes, plan, N, K, stream=stream),
                 lambda: mx.linear_experts_wgrad(x, x, plan, stream=stream)):
        with pytest.raises(ValueError, match="stream must be on cuda:0"):
            call()
