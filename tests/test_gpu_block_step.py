"""The operators between the GEMMs together with the GEMMs (the example that trains
an MLP block, its products against the oracle's), and every one of their kernels
in the bounds-checked build."""
import ctypes

import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
import oracle
from mxfp4_precision_gb300 import build
from tests.block_testutil import assert_near, canonical_scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


def test_training_an_mlp_block_reduces_its_loss():
    from examples.mlp_block_step import train
    losses, norms = train(report=lambda *_: None)
    assert np.isfinite(losses).all() and np.isfinite(norms).all()
    assert losses[-1] < 0.75 * losses[0]
    again, _ = train(report=lambda *_: None)
    assert again == losses                            # the same bits every time


def test_block_products_read_the_encoded_rows():
    """Both forward products of the block against the oracle's, on the operands that the norm and SwiGLU
    encoded."""
    from examples.mlp_block_step import MLPBlock
    T, K, F = 200, 256, 352
    b = MLPBlock(K, F, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, K, generator=g, device="cuda")
    r = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    out, (n, gu, a, w_gu, w_d) = b.forward(x, r)
    mx.check_status()
    for got, o, w, k in ((gu, n, w_gu, K), (out, a, w_d, F)):
        q, s = oracle.quantize(w.view(torch.int16).cpu().numpy().view(np.uint16), oracle.CONTRACT_COLS)
        ref, mag = oracle.gemm(o.codes.cpu().numpy(), canonical_scales(o.scales.cpu().numpy(), T, k)[0], q, s)
        assert_near(got, ref, 1e-5 * mag, "product")


# --------------------------------------------------------------------------- bounds-checked build
def _buf(n):
    # exact-size buffers, so that any overrun leaves the allocation
    return torch.full((max(1, n),), 0xA5, dtype=torch.uint8, device="cuda")


def _x(rows, cols, f32, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return x if f32 else x.bfloat16()


@pytest.fixture(scope="module")
def libs():
    normal, checked = mx.lib(), ctypes.CDLL(build.build(checked=True))
    for name in ("mx_rmsnorm", "mx_rmsnorm_backward", "mx_swiglu", "mx_swiglu_backward", "mx_clip_grads",
                 "mx_check_status"):
        getattr(checked, name).argtypes = getattr(normal, name).argtypes
    return normal, checked


def _same(outs):
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,K", [(1, 32), (5, 1056), (130, 288), (3, 4128), (2500, 512), (2, 32768), (700, 2080)])
@pytest.mark.parametrize("xf,sf,fmt", [(1, 0, 2), (0, 0, 1), (0, 1, 2)])
def test_checked_norm_stays_in_bounds(libs, T, K, xf, sf, fmt):
    x, r, w = _x(T, K, xf, 1), _x(T, K, sf, 2), _x(1, K, 0, 3)
    dres, outs = _x(T, K, sf, 4), []
    for L in libs:
        h, y, codes = _buf(T * K * (4 if sf else 2)), _buf(T * K * 2), _buf(T * K * fmt // 2)
        scales, rstd = _buf(mx.scales_bytes(T, K)), torch.zeros(T, device="cuda")
        assert L.mx_rmsnorm(x.data_ptr(), xf, K, r.data_ptr(), sf, K, w.data_ptr(), 0, 1e-5, T, K, h.data_ptr(), K,
                            y.data_ptr(), fmt, codes.data_ptr(), scales.data_ptr(), rstd.data_ptr(), None) == 0
        dx, dw = _buf(T * K * (4 if sf else 2)), _buf(4 * K)
        n = mx.rmsnorm_backward_workspace_bytes(T, K)
        ws = _buf(n)
        assert L.mx_rmsnorm_backward(x.data_ptr(), xf, K, h.data_ptr(), sf, K, w.data_ptr(), 0, rstd.data_ptr(),
                                     dres.data_ptr(), K, T, K, dx.data_ptr(), K, dw.data_ptr(), ws.data_ptr(), n,
                                     None) == 0
        assert L.mx_check_status(None) == 0
        outs.append((h, y, codes, scales, rstd, dx, dw))
    _same(outs)


@pytest.mark.parametrize("T,K,sf", [(4901, 512, 0), (4865, 1280, 1), (700, 4096, 0), (320, 6144, 0), (170, 16384, 0)])
def test_checked_norm_gradient_of_many_rows_stays_in_bounds(libs, T, K, sf):
    dy, h, w = _x(T, K, 1 - sf, 11), _x(T, K, sf, 12), _x(1, K, 0, 13)
    rstd, outs = torch.rand(T, device="cuda"), []
    for L in libs:
        dx, dw = _buf(T * K * (4 if sf else 2)), _buf(4 * K)
        n = mx.rmsnorm_backward_workspace_bytes(T, K)
        ws = _buf(n)
        assert L.mx_rmsnorm_backward(dy.data_ptr(), 1 - sf, K, h.data_ptr(), sf, K, w.data_ptr(), 0, rstd.data_ptr(),
                                     h.data_ptr(), K, T, K, dx.data_ptr(), K, dw.data_ptr(), ws.data_ptr(), n,
                                     None) == 0
        assert L.mx_check_status(None) == 0
        outs.append((dx, dw))
    _same(outs)


@pytest.mark.parametrize("T,F", [(1, 32), (5, 1056), (130, 288), (3, 4128), (700, 2080)])
@pytest.mark.parametrize("gf,fmt", [(1, 2), (0, 1)])
def test_checked_swiglu_stays_in_bounds(libs, T, F, gf, fmt):
    gu, dy, outs = _x(T, 2 * F, gf, 5), _x(T, F, 1 - gf, 6), []
    for L in libs:
        y, codes, scales, d = _buf(T * F * 2), _buf(T * F * fmt // 2), _buf(mx.scales_bytes(T, F)), _buf(T * F * 4)
        assert L.mx_swiglu(gu.data_ptr(), gf, 2 * F, T, F, y.data_ptr(), fmt, codes.data_ptr(), scales.data_ptr(),
                           None) == 0
        assert L.mx_swiglu_backward(dy.data_ptr(), 1 - gf, F, gu.data_ptr(), gf, 2 * F, T, F, d.data_ptr(), None) == 0
        assert L.mx_check_status(None) == 0
        outs.append((y, codes, scales, d))
    _same(outs)


@pytest.mark.parametrize("sizes", [[1], [7, 8192, 8193, 3, 100001], [5] * 100, [1 << 22]])
@pytest.mark.parametrize("gf,of,skew", [(1, 0, 0), (0, 0, 1), (1, 1, 1)])
def test_checked_clip_stays_in_bounds(libs, sizes, gf, of, skew):
    gs, outs = [_x(1, n, gf, 7).view(-1) for n in sizes], []
    for L in libs:
        to = [torch.zeros(n + skew, dtype=torch.float32 if of else torch.bfloat16, device="cuda") for n in sizes]
        n = len(sizes)
        arr = lambda t, v: (t * n)(*v)  # noqa: E731
        norm, need = torch.zeros(1, device="cuda"), mx.grad_workspace_bytes(n)
        ws = _buf(need)
        assert L.mx_clip_grads(arr(ctypes.c_void_p, [g.data_ptr() for g in gs]), arr(ctypes.c_int64, sizes),
                               arr(ctypes.c_int, [gf] * n),
                               arr(ctypes.c_void_p, [t[skew:].data_ptr() for t in to]), arr(ctypes.c_int, [of] * n),
                               n, 0.5, 1e-6, norm.data_ptr(), ws.data_ptr(), need, None) == 0
        assert L.mx_check_status(None) == 0
        outs.append((norm, *to))
        assert not any(t[:skew].any() for t in to)
    _same(outs)
