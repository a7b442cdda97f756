"""The operators between the GEMMs (mx_rmsnorm, mx_swiglu, their gradients,
mx_grad_norm, mx_clip_grads) against plain forms in 64 bits, on odd and ragged
sizes, every type, pitches, in-place forms, rows of zeros, Inf and NaN,
streams, graph capture and offsets beyond 32 bits.  The tolerances are
derived in block_testutil.py; gradients are checked against the formula and
against differences of the 64-bit forward form."""
import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
import oracle
from tests.block_testutil import (DELTA, TINY, U, UB, assert_encoded, assert_near, canonical_scales,
                                  f64, norm64, norm_backward64, sigmoid64, swiglu64,
                                  swiglu_backward64)

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mxfp4_precision_gb300 import build
    build.build()
    mx.lib()


def _matrix(rows, cols, dtype, seed, pad=0, std=1.0):
    """Normal values with a few large columns; a slice of a wider matrix if pad."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda") * std
    x[:, ::37] *= 20
    return x.to(dtype)[:, :cols]


def _weight(n, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(dtype)


def _rounding(dtype):
    return UB if dtype == BF16 else 0.0


# --------------------------------------------------------------------------- norm
NORM_SIZES = [(1, 32), (1, 4096), (3, 64), (5, 96), (129, 256), (130, 288), (33, 1056), (7, 4128),
              (2, 8192), (3, 16384), (2, 32768), (257, 2080), (64, 5120)]


@pytest.mark.parametrize("T,K", NORM_SIZES)
@pytest.mark.parametrize("xt,st,wt,fmt,pad", [
    (F32, BF16, BF16, "mx8", 0), (BF16, BF16, BF16, "mx4", 32), (BF16, F32, F32, "mx8", 8),
    (F32, F32, BF16, None, 64)])
def test_norm_with_residual(T, K, xt, st, wt, fmt, pad):
    x, r, w = _matrix(T, K, xt, 1, pad), _matrix(T, K, st, 2, pad, 2.0), _weight(K, wt, 3)
    f = {"mx8": mx.FMT_MXFP8, "mx4": mx.FMT_MXFP4, None: None}[fmt]
    o = mx.rmsnorm(x, w, residual=r, eps=EPS, fmt=f)
    mx.check_status()
    h, y, rstd = norm64(f64(x), f64(r), f64(w), EPS)
    assert o.h.dtype == st and o.h.is_contiguous()
    assert_near(o.h, h, np.abs(h) * _rounding(st) + 2 * U * (np.abs(f64(x)) + np.abs(f64(r))), "h")
    assert_near(o.rstd, rstd, rstd * DELTA, "rstd")
    # h's own rounding in fp32 is relative to |x| + |r|, not to their sum
    slack = 2 * U * (np.abs(f64(x)) + np.abs(f64(r))) * rstd[:, None] * np.abs(f64(w))
    assert_near(o.y, y, np.abs(y) * (UB + DELTA) + slack + TINY, "y")
    if fmt is None:
        assert o.codes is None and o.scales is None
        return
    y32 = (x.float() + r.float()).double().cpu().numpy()    # fp32's h: the encoder's input is exact in it
    assert_encoded(o.codes, o.scales, y32 * rstd[:, None] * f64(w), f, fmt == "mx8", f"{T}x{K}")


@pytest.mark.parametrize("T,K", [(2433, 768), (2440, 1024), (2432, 1280), (2435, 2080), (2432, 4128), (2432, 8192)])
@pytest.mark.parametrize("xt,st,fmt", [(F32, BF16, "mx8"), (BF16, BF16, "mx4"), (F32, F32, "mx8")])
def test_norm_many_rows(T, K, xt, st, fmt):
    """Rows enough to fill the SMs: the ways of cutting a row that only then are taken."""
    test_norm_with_residual(T, K, xt, st, BF16, fmt, 0)


@pytest.mark.parametrize("T,K", [(1, 8), (4, 40), (3, 1000), (129, 72), (2, 24), (5, 32760)])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_norm_without_residual_any_multiple_of_8(T, K, xt):
    x, w = _matrix(T, K, xt, 4), _weight(K, BF16, 5)
    o = mx.rmsnorm(x, w, eps=EPS)
    mx.check_status()
    _, y, rstd = norm64(f64(x), None, f64(w), EPS)
    assert o.h is None and o.codes is None
    assert_near(o.y, y, np.abs(y) * (UB + DELTA) + TINY, "y")
    assert_near(o.rstd, rstd, rstd * DELTA, "rstd")


def test_norm_only_the_operand_and_the_empty_batch():
    x, w = _matrix(5, 512, BF16, 6), _weight(512, BF16, 7)
    a, b = mx.rmsnorm(x, w, fmt=mx.FMT_MXFP8, want_y=False), mx.rmsnorm(x, w, fmt=mx.FMT_MXFP8)
    mx.check_status()
    assert a.y is None and torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    o = mx.rmsnorm(x[:0], w, residual=x[:0], fmt=mx.FMT_MXFP8)
    assert o.y.shape == (0, 512) and o.codes.shape == (0, 512)
    dx, dw = mx.rmsnorm_backward(x[:0], x[:0], w, o.rstd)
    mx.check_status()
    assert dx.shape == (0, 512) and not dw.any()


def test_norm_in_place_matches_out_of_place():
    for dtype in (BF16, F32):
        x, r, w = _matrix(130, 1056, F32, 8), _matrix(130, 1056, dtype, 9, 32), _weight(1056, BF16, 10)
        a = mx.rmsnorm(x, w, residual=r, fmt=mx.FMT_MXFP8)
        b = mx.rmsnorm(x, w, residual=r, fmt=mx.FMT_MXFP8, out_h=r)
        mx.check_status()
        assert b.h is r and torch.equal(a.h, r)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def test_norm_zero_inf_and_nan_rows():
    K = 512
    x = _matrix(6, K, F32, 11)
    x[1] = 0
    x[2, 40] = float("nan")
    x[3, 100] = float("inf")
    x[4] = 1e-30
    x[5, :32] = 0
    w = _weight(K, F32, 12)
    o = mx.rmsnorm(x, w, eps=EPS, fmt=mx.FMT_MXFP8)
    mx.check_status()
    s, clean = canonical_scales(o.scales.cpu().numpy(), 6, K)
    codes, y = o.codes.cpu().numpy(), f64(o.y)
    assert clean
    assert not y[1].any() and not codes[1].any() and not s[1].any()
    # a NaN reaches rstd and so the whole row: every block marked, codes zero
    assert np.isnan(y[2]).all() and (s[2] == 0xFF).all() and not codes[2].any()
    # Inf: rstd = 0, Inf * 0 is NaN in its own block alone, 0 elsewhere
    assert np.isnan(y[3, 100]) and not y[3, :100].any() and not y[3, 101:].any()
    assert s[3, 3] == 0xFF and not np.delete(s[3], 3).any()
    assert not codes[3, 96:128].any() and not (codes[3] & 0x7F).any()   # signed zeros beside it
    assert_near(o.y[4:5], norm64(f64(x[4:5]), None, f64(w), EPS)[1], 1e-27 * (UB + DELTA) + 1e-29, "tiny row")
    assert s[5, 0] == 0 and not codes[5, :32].any() and codes[5, 32:].any()


def test_norm_operand_feeds_the_gemm():
    """The encoded rows are the operand that mx_gemm_mxfp8 / mx_gemm read."""
    T, K, N = 200, 512, 136
    x, w = _matrix(T, K, BF16, 13), _weight(K, BF16, 14)
    B = _matrix(K, N, BF16, 15, std=0.02)
    o = mx.rmsnorm(x, w, fmt=mx.FMT_MXFP8)
    Bq, Bs = mx.quantize_mxfp8(B)
    C = mx.gemm_mxfp8(o.codes, o.scales, Bq, Bs, T, N, K)
    o4 = mx.rmsnorm(x, w, fmt=mx.FMT_MXFP4)
    B4, B4s = mx.quantize(B, mx.CONTRACT_ROWS)
    C4 = mx.gemm(o4.codes, o4.scales, B4, B4s, T, N, K)
    mx.check_status()
    for out, got, (q, s), fmt in ((C, o, (Bq, Bs), oracle.FMT_MXFP8), (C4, o4, (B4, B4s), oracle.FMT_MXFP4)):
        As, _ = canonical_scales(got.scales.cpu().numpy(), T, K)
        Bc, _ = canonical_scales(s.cpu().numpy()[:mx.scales_bytes(N, K)], N, K)
        ref, mag = oracle.gemm(got.codes.cpu().numpy(), As, q.cpu().numpy(), Bc, fmt)
        assert_near(out, ref, 1e-5 * mag, "gemm of the encoded rows")


@pytest.mark.parametrize("T,K", [(1, 32), (1, 4096), (3, 8), (97, 2080), (130, 1000), (700, 264),
                                 (5, 8192), (3, 16384), (2, 32768), (1300, 1056)])
@pytest.mark.parametrize("dt,st,wt,pad,res", [(F32, BF16, BF16, 0, True), (BF16, BF16, F32, 8, True),
                                              (BF16, F32, BF16, 0, False), (F32, F32, F32, 32, True)])
def test_norm_backward(T, K, dt, st, wt, pad, res):
    dy, h, w = _matrix(T, K, dt, 21, pad, 1e-3), _matrix(T, K, st, 22, pad), _weight(K, wt, 23)
    dres = _matrix(T, K, st, 24, pad, 1e-3) if res else None
    rstd = torch.from_numpy(norm64(f64(h), None, f64(w), EPS)[2]).float().cuda()
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    mx.check_status()
    d64, h64, w64, r64 = f64(dy), f64(h), f64(w), f64(rstd)
    g64 = None if dres is None else f64(dres)
    rx, rw = norm_backward64(d64, h64, w64, r64, g64)
    a, xh = d64 * w64, h64 * r64[:, None]
    size = r64[:, None] * (np.abs(a) + np.abs(xh) * np.abs(a * xh).mean(-1, keepdims=True))
    size += 0 if g64 is None else np.abs(g64)
    assert dx.dtype == st
    assert_near(dx, rx, np.abs(rx) * _rounding(st) + DELTA * size + TINY, "dx")
    # a column's sum over T rows: at most T roundings in a chain
    assert_near(dw, rw, (T + 16) * U * np.abs(d64 * xh).sum(0) + TINY, "dw")
    again = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    mx.check_status()
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


# Rows enough for the ring, at every way of cutting a row there.
RING_SIZES = [(4900, 256), (4901, 512), (4900, 760), (4864, 1024), (4865, 1280), (800, 2048), (700, 4096), (620, 5120),
              (320, 6144), (311, 8192), (170, 16384)]


@pytest.mark.parametrize("T,K", RING_SIZES)
@pytest.mark.parametrize("dt,st,pad,res", [(F32, BF16, 0, True), (BF16, BF16, 8, False), (F32, F32, 0, True)])
def test_norm_backward_many_rows(T, K, dt, st, pad, res):
    test_norm_backward(T, K, dt, st, BF16, pad, res)


@pytest.mark.parametrize("T", [3, 170])
def test_norm_backward_just_beyond_16384_columns(T):
    test_norm_backward(T, 17024, BF16, BF16, BF16, 0, True)


def _skewed(t):
    """The same matrix at 16 bytes off a 32-byte boundary."""
    wide = torch.zeros(t.shape[0], t.shape[1] + 16, dtype=t.dtype, device="cuda")
    skew = 16 // t.element_size()
    wide[:, skew:skew + t.shape[1]] = t
    return wide[:, skew:skew + t.shape[1]]


@pytest.mark.parametrize("T,K", [(5, 4096), (700, 2080)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_off_a_32_byte_boundary_give_the_same_bits(T, K, dtype):
    x, r, w, dres = (_matrix(T, K, dtype, 91), _matrix(T, K, dtype, 92), _weight(K, F32, 93), _matrix(T, K, dtype, 94))
    gu, dy = _matrix(T, 2 * K, dtype, 95), _matrix(T, K, dtype, 96)
    runs = []
    for f in (lambda t: t, _skewed):
        o = mx.rmsnorm(f(x), w, residual=f(r), fmt=mx.FMT_MXFP8, out_h=f(torch.zeros_like(r)))
        dx, dw = mx.rmsnorm_backward(f(dy), f(x), w, o.rstd, dres=f(dres), out_dx=f(torch.zeros_like(r)))
        g = mx.swiglu(f(gu), fmt=mx.FMT_MXFP8)
        runs.append([*o, dx, dw, *g, mx.swiglu_backward(f(dy), f(gu))])
    mx.check_status()
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_norm_backward_in_place_many_rows():
    T, K = 700, 4096
    dy, h, w = _matrix(T, K, BF16, 35), _matrix(T, K, BF16, 36), _weight(K, F32, 37)
    dres = _matrix(T, K, BF16, 38, 32)
    rstd = mx.rmsnorm(h, w).rstd
    a, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    b, dw2 = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres, out_dx=dres)
    mx.check_status()
    assert torch.equal(a, b) and torch.equal(dw, dw2)
    a, _ = mx.rmsnorm_backward(dy, h, w, rstd)
    b, none = mx.rmsnorm_backward(dy, h, w, rstd, want_dw=False, out_dx=dy)
    mx.check_status()
    assert none is None and torch.equal(a, b)


def test_norm_backward_in_place_and_without_dw():
    dy, h, w = _matrix(70, 1056, F32, 25), _matrix(70, 1056, BF16, 26), _weight(1056, BF16, 27)
    dres = _matrix(70, 1056, BF16, 28, 32)
    rstd = mx.rmsnorm(h, w).rstd
    a, dw = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres)
    b, none = mx.rmsnorm_backward(dy, h, w, rstd, dres=dres, want_dw=False, out_dx=dres)
    mx.check_status()
    assert none is None and b is dres and torch.equal(a, b)
    hf = h.float()
    a, _ = mx.rmsnorm_backward(dy, hf, w, rstd)
    b, _ = mx.rmsnorm_backward(dy, hf, w, rstd, out_dx=dy)
    mx.check_status()
    assert b is dy and torch.equal(a, b)


def test_norm_gradient_against_differences():
    """d/dt of sum(v * y(h + t d)) by central differences of the 64-bit form, with the step's
    truncation (third derivative, O(t^2)) far below the kernel's DELTA."""
    T, K = 9, 352
    h, w, v = _matrix(T, K, F32, 31), _weight(K, F32, 32), _matrix(T, K, F32, 33)
    rstd = mx.rmsnorm(h, w, eps=EPS).rstd
    dx, dw = mx.rmsnorm_backward(v, h, w, rstd)
    mx.check_status()
    g = np.random.default_rng(34)
    h64, w64, v64, t = f64(h), f64(w), f64(v), 1e-4
    for _ in range(4):
        d = g.standard_normal((T, K))
        y = [(v64 * norm64(h64 + s * t * d, None, w64, EPS)[1]).sum(-1) for s in (-1, 1)]
        assert_near((f64(dx) * d).sum(-1), (y[1] - y[0]) / (2 * t),
                    4 * DELTA * np.abs(v64 * w64 * d).sum(-1) * f64(rstd), "dx along d")
        d = g.standard_normal(K)
        y = [v64 * norm64(h64, None, w64 + s * t * d, EPS)[1] for s in (-1, 1)]
        ref = ((y[1] - y[0]) / (2 * t)).sum(0)
        assert_near(f64(dw) * d, ref, 4 * DELTA * np.abs(v64 * h64 * f64(rstd)[:, None]).sum(0) * np.abs(d), "dw")


# --------------------------------------------------------------------------- SwiGLU
GLU_SIZES = [(1, 32), (1, 14336), (4, 64), (127, 96), (129, 288), (3, 4128), (35, 1760), (2, 40000)]


@pytest.mark.parametrize("T,F", GLU_SIZES)
@pytest.mark.parametrize("gt,fmt,pad", [(F32, "mx8", 0), (BF16, "mx8", 32), (BF16, "mx4", 0), (F32, "mx4", 8)])
def test_swiglu(T, F, gt, fmt, pad):
    gu = _matrix(T, 2 * F, gt, 41, pad)
    f = mx.FMT_MXFP8 if fmt == "mx8" else mx.FMT_MXFP4
    o = mx.swiglu(gu, fmt=f)
    mx.check_status()
    y = swiglu64(f64(gu))
    assert_near(o.y, y, np.abs(y) * (UB + DELTA) + TINY, "y")
    assert_encoded(o.codes, o.scales, y, f, fmt == "mx8", f"{T}x{F}")


@pytest.mark.parametrize("T,F", [(20003, 288), (10001, 1056)])
def test_swiglu_many_rows(T, F):
    """Rows enough for several to a thread."""
    test_swiglu(T, F, F32, "mx8", 0)
    test_swiglu(T, F, BF16, "mx4", 8)


@pytest.mark.parametrize("T,F", [(1, 8), (5, 24), (3, 1000)])
def test_swiglu_plain_any_multiple_of_8(T, F):
    gu = _matrix(T, 2 * F, F32, 42)
    o = mx.swiglu(gu)
    mx.check_status()
    y = swiglu64(f64(gu))
    assert o.codes is None
    assert_near(o.y, y, np.abs(y) * (UB + DELTA) + TINY, "y")


def test_swiglu_extremes():
    """Gates whose exponential overflows or vanishes, zeros, NaN and Inf."""
    g = torch.tensor([0.0, -0.0, 100.0, -100.0, 88.0, -88.0, 20.0, -20.0, 1e-30, -1e-30, 3e38, -3e38,
                      float("inf"), float("nan"), -1.278, 5.0] + [0.5] * 16, device="cuda")
    gu = torch.cat([g, torch.full((32,), 2.0, device="cuda")]).view(1, 64)
    dy = torch.full((1, 32), 0.5, device="cuda")
    o = mx.swiglu(gu, fmt=mx.FMT_MXFP8)
    d = mx.swiglu_backward(dy, gu)
    mx.check_status()
    y, d = f64(o.y)[0], f64(d)[0]
    fin = np.r_[0:12, 14:32]
    want = swiglu64(f64(gu))[0]
    big = np.abs(want) > 3.39e38                      # 2 * 3e38 overflows to Inf in any 32-bit form
    assert np.isinf(y[10]) and big[10]
    k = fin[fin != 10]
    # beyond exp's range the sigmoid is 0 in fp32: an absolute error of its smallest value times |g u|
    assert_near(y[k], want[k], np.abs(want[k]) * (UB + DELTA) + 1e-36, "y")
    assert np.isinf(y[12]) and np.isnan(y[13])
    assert o.scales[0] == 0xFF and not o.codes.any()
    ref = swiglu_backward64(f64(dy), f64(gu))[0]
    s = sigmoid64(f64(gu)[0, :32])
    gg = f64(gu)[0, :32]
    k = fin[(fin != 10) & (fin != 11)]
    assert_near(d[k], ref[k], np.abs(ref[k]) * UB + DELTA * np.abs(s[k]) * (1 + np.abs(gg[k] * (1 - s[k]))) + 1e-35, "dg")
    assert_near(d[32 + k], ref[32 + k], np.abs(ref[32 + k]) * (UB + DELTA) + 1e-35, "du")
    assert np.isnan(d[13]) and np.isnan(d[45])


@pytest.mark.parametrize("T,F", [(1, 8), (1, 14336), (333, 1760), (5, 24), (130, 1000), (3, 4128)])
@pytest.mark.parametrize("dt,gt,pad", [(F32, F32, 0), (BF16, BF16, 8), (F32, BF16, 32), (BF16, F32, 0)])
def test_swiglu_backward(T, F, dt, gt, pad):
    dy, gu = _matrix(T, F, dt, 51, pad, 1e-3), _matrix(T, 2 * F, gt, 52, pad)
    d = mx.swiglu_backward(dy, gu)
    mx.check_status()
    ref = swiglu_backward64(f64(dy), f64(gu))
    g, u = np.split(f64(gu), 2, -1)
    s = sigmoid64(g)
    size = np.concatenate([np.abs(f64(dy) * u) * s * (1 + np.abs(g) * (1 - s)), np.abs(f64(dy) * g) * s], -1)
    assert_near(d, ref, np.abs(ref) * UB + DELTA * size + TINY, "dgu")


def test_swiglu_gradient_against_differences():
    T, F = 7, 96
    gu, v = _matrix(T, 2 * F, F32, 53), _matrix(T, F, F32, 54)
    d = f64(mx.swiglu_backward(v, gu))
    mx.check_status()
    g64, v64, t = f64(gu), f64(v), 1e-5
    rng = np.random.default_rng(55)
    for _ in range(4):
        e = rng.standard_normal((T, 2 * F))
        y = [(v64 * swiglu64(g64 + s * t * e)).sum(-1) for s in (-1, 1)]
        ref = (y[1] - y[0]) / (2 * t)
        # dgu is rounded to bf16: half an ulp of each product; the difference's own error is far below
        assert_near((d * e).sum(-1), ref, 2 * UB * np.abs(d * e).sum(-1) + 1e-6 * np.abs(ref), "dgu along e")


# --------------------------------------------------------------------------- clipping
def _grads(sizes, dtype, seed, std=0.02):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(dtype) for n in sizes]


def _norm64(ts):
    return float(np.sqrt(sum((f64(t) ** 2).sum() for t in ts)))


ODD = [1, 3, 8, 17, 4096, 8191, 8192, 8193, 100003, 0, 5, 65536]


@pytest.mark.parametrize("sizes", [[1], [7], [8192], ODD, [33] * 70, [5] * 1030, [1 << 21, 3, 1 << 20]])
@pytest.mark.parametrize("dt,ot", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("std", [0.02, 1e-7])
def test_clip_into_a_flat_bucket(sizes, dt, ot, std):
    """Outputs are slices of one bucket, at any element's alignment; what lies between stays."""
    gs = _grads(sizes, dt, 61, std)
    flat = torch.full((sum(sizes) + 2 * len(sizes) + 1,), 7.0, dtype=ot, device="cuda")
    outs, at = [], 1
    for n in sizes:
        outs.append(flat[at:at + n])
        at += n + 2
    keep = [g.clone() for g in gs]
    norm = mx.clip_grads(gs, 0.01, out=outs)
    only = mx.grad_norm(gs)
    mx.check_status()
    n64 = _norm64(keep)
    assert_near(f64(norm), np.array([n64]), n64 * 2.0 ** -22, "norm")
    assert torch.equal(norm, only)
    coef = min(1.0, 0.01 / (n64 + 1e-6))
    for g, k, o in zip(gs, keep, outs):
        assert torch.equal(g, k)
        ref = f64(k) * coef
        assert_near(o, ref, np.abs(ref) * (_rounding(ot) + DELTA) + TINY, "clipped")
    gaps = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    at = 1
    for n in sizes:
        gaps[at:at + n] = False
        at += n + 2
    assert (flat[gaps] == 7.0).all()


@pytest.mark.parametrize("count", [63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 2049])
def test_clip_at_the_edges_of_the_table(count):
    """As many tensors as one table holds, one fewer and one more; 1 to 40 elements each."""
    gs = _grads([1 + (7 * i) % 40 for i in range(count)], F32, 67)
    n64 = _norm64(gs)
    refs = [f64(g) * (0.01 / (n64 + 1e-6)) for g in gs]
    norm = mx.clip_grads(gs, 0.01)
    mx.check_status()
    assert_near(f64(norm), np.array([n64]), n64 * 2.0 ** -22, "norm")
    for g, ref in zip(gs, refs):
        assert_near(g, ref, np.abs(ref) * (_rounding(F32) + DELTA) + TINY, "clipped")


@pytest.mark.parametrize("dt", [F32, BF16])
def test_clip_in_place_and_unaligned(dt):
    base = _grads([50000], dt, 62)[0]
    gs = [base[1:7], base[9:4100], base[4100:4100], base[4103:40000], base[40008:]]
    ref = base.clone()
    outs = [torch.empty_like(g) for g in gs]
    n0 = mx.clip_grads(gs, 0.5, out=outs)
    n1 = mx.clip_grads(gs, 0.5)
    mx.check_status()
    assert torch.equal(n0, n1) and float(n0) > 0.5
    for g, o in zip(gs, outs):
        assert torch.equal(g, o)
    untouched = torch.ones(base.numel(), dtype=torch.bool, device="cuda")
    for a, b in ((1, 7), (9, 4100), (4103, 40000), (40008, 50000)):
        untouched[a:b] = False
    assert torch.equal(base[untouched], ref[untouched])
    kept = base.clone()
    mx.clip_grads(gs, 100.0)                          # nothing to clip: the same bits
    mx.check_status()
    assert torch.equal(base, kept)


def test_clip_mixed_types_and_layer_sizes():
    gs = _grads([4096 * 1024, 4096], F32, 63) + _grads([1024 * 512 + 4, 3], BF16, 64)
    n64 = _norm64(gs)
    keep = [f64(g) for g in gs]
    norm = mx.clip_grads(gs, 1.0)
    mx.check_status()
    assert_near(f64(norm), np.array([n64]), n64 * 2.0 ** -22, "norm")
    for g, k in zip(gs, keep):
        ref = k / (n64 + 1e-6)
        assert_near(g, ref, np.abs(ref) * (_rounding(g.dtype) + DELTA) + TINY, "clipped")


def test_clip_empty_zero_nan_and_inf():
    assert float(mx.grad_norm([])) == 0.0
    assert float(mx.clip_grads([torch.empty(0, device="cuda")], 1.0)) == 0.0
    z = torch.zeros(1000, device="cuda")
    assert float(mx.clip_grads([z], 1.0)) == 0.0 and not z.any()
    g = torch.ones(1000, device="cuda")
    g[3] = float("inf")
    n = mx.clip_grads([g], 1.0)
    assert torch.isinf(n).all() and torch.isnan(g[3]) and not g[4:].any()
    g = torch.ones(1000, device="cuda")
    g[3] = float("nan")
    n = mx.clip_grads([g], 1.0)
    mx.check_status()
    assert torch.isnan(n).all() and torch.isnan(g).all()
    g = torch.ones(16, device="cuda")
    mx.clip_grads([g], 0.0)
    mx.check_status()
    assert not g.any()


# --------------------------------------------------------------------------- streams, graphs, large offsets
def test_other_stream_and_graph_capture():
    T, K = 300, 1056
    x, r, w = _matrix(T, K, F32, 71), _matrix(T, K, BF16, 72), _weight(K, BF16, 73)
    gu = _matrix(T, 2 * K, BF16, 74)
    gs = _grads(ODD, F32, 75)
    outs = [torch.empty_like(g) for g in gs]

    def all_of(stream=None):
        a = mx.rmsnorm(x, w, residual=r, fmt=mx.FMT_MXFP8, stream=stream)
        dx, dw = mx.rmsnorm_backward(x, a.h, w, a.rstd, dres=r, stream=stream)
        b = mx.swiglu(gu, fmt=mx.FMT_MXFP4, stream=stream)
        d = mx.swiglu_backward(a.y, gu, stream=stream)
        n = mx.clip_grads(gs, 0.5, out=outs, stream=stream)
        return [*a, dx, dw, *b, d, n, *outs]
    ref = [t.clone() for t in all_of()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(side)
    side.synchronize()
    mx.check_status(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for t in got:
        t.zero_()
    graph.replay()
    mx.check_status()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_offsets_beyond_32_bits():
    """Matrices and a gradient of more than 2^31 elements: the last rows and elements are right."""
    T, K = 65537, 32768
    x = torch.zeros((T, K), dtype=BF16, device="cuda")
    x[-3:] = _matrix(3, K, BF16, 81)
    w = _weight(K, BF16, 82)
    o = mx.rmsnorm(x, w, fmt=mx.FMT_MXFP8)
    mx.check_status()
    small = mx.rmsnorm(x[-3:].clone(), w, fmt=mx.FMT_MXFP8)
    assert torch.equal(o.y[-3:], small.y) and torch.equal(o.codes[-3:], small.codes)
    assert not (o.codes[:1000] & 0x7F).any()           # zeros, negative under a negative weight
    dx, dw = mx.rmsnorm_backward(x, x, w, o.rstd)
    dx3, dw3 = mx.rmsnorm_backward(x[-3:].clone(), x[-3:].clone(), w, small.rstd)
    mx.check_status()
    assert torch.equal(dx[-3:], dx3)
    assert_near(dw, f64(dw3), np.abs(f64(dw3)) * DELTA + 1e-3, "dw")
    del o, dx
    y = mx.swiglu(x)
    y3 = mx.swiglu(x[-3:].clone())
    d = mx.swiglu_backward(y.y, x)
    mx.check_status()
    assert torch.equal(y.y[-3:], y3.y)
    assert torch.equal(d[-3:], mx.swiglu_backward(y3.y, x[-3:].clone()))
    del y, d
    flat = x.view(-1)
    out = torch.empty(flat.numel(), dtype=BF16, device="cuda")
    n = mx.clip_grads([flat], 1.0, out=[out])
    mx.check_status()
    n64 = _norm64([flat[-3 * K:]])
    assert_near(f64(n), np.array([n64]), n64 * 2.0 ** -22, "norm")
    ref = f64(flat[-3 * K:]) / (n64 + 1e-6)
    assert_near(out[-3 * K:], ref, np.abs(ref) * (UB + DELTA) + TINY, "clipped")
