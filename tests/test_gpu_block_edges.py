"""The operators between the GEMMs where their values are easily lost: the bits of
SwiGLU's fp32 formula, gates beyond 80 and elements beside them, the scales' padding of rows
that hold no numbers, gradients and outputs at every alignment."""
import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
import oracle
from tests.block_testutil import (DELTA, TINY, UB, assert_near, canonical_scales, f64, sigmoid64, swiglu64,
                                  swiglu_backward64)

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mxfp4_precision_gb300 import build
    build.build()
    mx.lib()


def _normal(rows, cols, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device="cuda") * std


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF16 else torch.int32)


# --------------------------------------------------------------------------- norm
@pytest.mark.parametrize("K", [32, 288, 1056, 4128])
@pytest.mark.parametrize("fmt", [mx.FMT_MXFP8, mx.FMT_MXFP4])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_scale_padding_is_zero_beside_rows_without_numbers(K, fmt, residual):
    """Rows whose rstd is NaN (a NaN in them), 0 (an Inf) or Inf (all zeros, eps = 0): their blocks are
    marked as the formula has them, the padding beyond K stays zero, and so do the rows between."""
    x = _normal(7, K, 21)
    x[1, 3] = float("nan")
    x[2, K - 1] = float("inf")
    x[4] = 0
    r = torch.zeros(7, K, dtype=BF16, device="cuda") if residual else None
    o = mx.rmsnorm(x, torch.ones(K, device="cuda"), residual=r, eps=0.0, fmt=fmt)
    mx.check_status()
    scales, clean = canonical_scales(o.scales.cpu().numpy(), 7, K)
    codes = o.codes.cpu().numpy()
    assert clean
    for row in (1, 4):
        assert (scales[row] == 0xFF).all() and not codes[row].any()
    assert scales[2, -1] == 0xFF and not scales[2, :-1].any()
    for row in (0, 3, 5, 6):
        assert codes[row].any() and (scales[row] != 0xFF).all()


# --------------------------------------------------------------------------- SwiGLU
def _gates(T, F, seed):
    """Rows of normal gates, then rows whose magnitudes spread over all of fp32 up to 80 (zeros of both
    signs and subnormals among them)."""
    g = _normal(T, F, seed, 3.0)
    r = torch.Generator(device="cuda").manual_seed(seed + 1)
    top = int(np.float32(80.0).view(np.int32))
    wide = torch.randint(0, top + 1, (T // 4, F), generator=r, device="cuda", dtype=torch.int32)
    wide[0, :8] = 0
    wide = wide.view(F32) * torch.where(torch.rand(T // 4, F, generator=r, device="cuda") < 0.5, -1.0, 1.0)
    g[-(T // 4):] = wide
    return g


@pytest.mark.parametrize("fmt", [mx.FMT_MXFP8, mx.FMT_MXFP4])
def test_swiglu_of_fp32_has_the_bits_of_the_formula(fmt):
    """y = g / (1 + exp(-g)) * u with every step rounded to fp32, then once to bf16 and once to the codes:
    no value, code or scale differs.  4M elements: a form that is off by an fp32 bit here and there
    moves some 6 in a million bf16 y across a rounding boundary."""
    T, F = 2048, 2048
    g, u = _gates(T, F, 1), _normal(T, F, 3)
    o = mx.swiglu(torch.cat([g, u], 1), fmt=fmt)
    mx.check_status()
    y = g / (1 + torch.exp(-g)) * u
    assert torch.equal(_bits(o.y), _bits(y.to(BF16)))
    fp8 = fmt == mx.FMT_MXFP8
    blocks = y.cpu().numpy().reshape(T, F // 32, 32)
    want = (oracle.scale_bytes_e4m3 if fp8 else oracle.scale_bytes)(np.abs(blocks).max(-1))
    scales, clean = canonical_scales(o.scales.cpu().numpy(), T, F)
    assert clean and np.array_equal(scales, want)
    # a power of two within fp32's range times a value: exact, or a zero of its sign in either format
    v = blocks * np.exp2(127.0 - want.astype(np.float64)).astype(np.float32)[..., None]
    c = (oracle.e4m3_rne if fp8 else oracle.e2m1_rne)(v).reshape(T, F)
    got = o.codes.cpu().numpy()
    if not fp8:
        got = np.stack([got & 15, got >> 4], -1).reshape(T, F)
    assert np.array_equal(got, c)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("far", [-80.5, 81.0, -300.0, 1e30])
def test_swiglu_beside_far_gates_keeps_its_bits(dtype, far):
    """One gate in eight replaced by one beyond 80, where its u is 0: no other element, code or scale
    changes, forward or backward."""
    T, F = 1024, 2048
    gu, dy = _normal(T, 2 * F, 11, 3.0), _normal(T, F, 12)
    at = torch.zeros(F, dtype=torch.bool, device="cuda")
    at[5::8] = True
    gu[:, F:][:, at] = 0
    runs = []
    for value in (0.5, far):
        gu[:, :F][:, at] = value
        x = gu.to(dtype)
        o = mx.swiglu(x, fmt=mx.FMT_MXFP8)
        d = mx.swiglu_backward(dy.to(dtype), x)
        # the far elements' own results: zeros whose sign is the gate's, and du of the gate itself
        runs.append([o.y[:, ~at], o.codes[:, ~at], o.scales, d[:, :F][:, ~at], d[:, F:][:, ~at]])
    mx.check_status()
    for a, b in zip(*runs):
        assert torch.equal(_bits(a) if a.dtype == BF16 else a, _bits(b) if b.dtype == BF16 else b)


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_swiglu_of_far_gates_beside_large_values(gt, dt):
    """Gates from -80 to -98, where exp(-g) leaves fp32 but exp(g) times u, or u and dy, is a normal value.

    The exponential's argument g log2(e) is rounded at up to 2^8 (2^-17 ln 2 of the result, 89 u), its
    factor to fp32 (0.23 u |g|, 23 u), the hardware's 2^x adds 4 u and the products 4 u: 120 u of DELTA's
    128.  Below 2^-126 the sigmoid has steps of 2^-149, of which one may be lost."""
    F = 352
    g = torch.cat([torch.linspace(-80.0, -98.0, F - 8), torch.tensor([80.5, 81, 88, 89, 100, 1e3, 1e10, 3e38])])
    g = g.to(gt).cuda()
    g64 = f64(g)
    mag = 10.0 ** torch.linspace(20, 30, F)
    mag[-8:] = 1e-3
    sign = torch.where(torch.arange(F) % 3 == 0, -1.0, 1.0)
    gu = torch.cat([g, (mag * sign).cuda().to(gt)]).view(1, 2 * F)
    dy = mag.flip(0).clone()
    dy[-8:] = 1e-3
    dy = dy.cuda().to(dt).view(1, F)
    o, d = mx.swiglu(gu), f64(mx.swiglu_backward(dy, gu))
    mx.check_status()
    u64, d64, s = f64(gu)[:, F:], f64(dy), sigmoid64(g64)
    step = np.where(s < 2.0 ** -126, 2.0 ** -149, 0.0)
    y = swiglu64(f64(gu))
    dgu = swiglu_backward64(d64, f64(gu))
    for got, ref, lost, what in ((f64(o.y), y, np.abs(g64 * u64) * step, "y"),
                                 (d[:, :F], dgu[:, :F], np.abs(d64 * u64 * (1 + np.abs(g64))) * step, "dg"),
                                 (d[:, F:], dgu[:, F:], np.abs(d64 * g64) * step, "du")):
        assert (np.abs(ref) < 1e38).all() and (np.abs(ref[:, :-8]) > 2.0 ** -126).all(), what
        bound = np.abs(ref) * (UB + DELTA) + lost + TINY
        assert (bound[:, :-8] < 0.5 * np.abs(ref[:, :-8])).all(), f"{what}: a lost sigmoid would pass"
        assert_near(got, ref, bound, what)


# --------------------------------------------------------------------------- clipping
@pytest.mark.parametrize("n", [5, 300, 5000])
@pytest.mark.parametrize("dt,ot", [(F32, BF16), (F32, F32), (BF16, F32), (BF16, BF16)])
def test_clip_at_every_pair_of_alignments(n, dt, ot):
    """Gradients that begin 0 to 8 elements off a 32-byte boundary into outputs that begin 0 to 8 off
    one (an fp32 gradient 4 off and a bf16 output 0 off are both 16-byte aligned), in one call."""
    pairs = [(a, b) for a in range(9) for b in range(9)]
    wide = -(-(n + 8) // 16) * 16 + 16
    x = _normal(len(pairs), wide, 31, 0.02).to(dt)
    out = torch.full((len(pairs), wide), 7.0, dtype=ot, device="cuda")
    grads = [x[i, a:a + n] for i, (a, _) in enumerate(pairs)]
    outs = [out[i, b:b + n] for i, (_, b) in enumerate(pairs)]
    norm = mx.clip_grads(grads, 0.1, out=outs)
    mx.check_status()
    want = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    assert_near(f64(norm), np.array([want]), want * 2.0 ** -22, "norm")
    assert want > 0.2
    gaps = torch.ones_like(out, dtype=torch.bool)
    for i, (a, b) in enumerate(pairs):
        ref = f64(grads[i]) * (0.1 / (want + 1e-6))
        assert_near(outs[i], ref, np.abs(ref) * (DELTA + (UB if ot == BF16 else 0)) + TINY, f"{a} -> {b}")
        gaps[i, b:b + n] = False
    assert (out[gaps] == 7.0).all()
