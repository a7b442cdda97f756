"""Products with bias, activation and residual in their epilogue, and their
gradient, against 64-bit forms; tolerances in product_testutil."""
import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.product_testutil import (ACTS, U, UB, Operand, act64, act_bound, assert_encoding_of, assert_output, assert_within, dev,
                                    epilogue64, f64, slope64)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FMT = {False: mx.FMT_MXFP4, True: mx.FMT_MXFP8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


def _vector(n, dtype, seed):
    return (torch.randn(n, generator=torch.Generator().manual_seed(seed)) * 4).to(dtype).cuda()


def _matrix(rows, cols, dtype, seed, pad=0, spread=4.0):
    x = torch.randn(rows, cols + pad, generator=torch.Generator().manual_seed(seed)) * spread
    return x.to(dtype).cuda()[:, :cols]


def _run(M, N, K, fp8, act="none", bias=None, res=None, seed=0, scale=-2, **kw):
    a, b = Operand(M, K, fp8, 2 * seed + 1, scale=scale), Operand(N, K, fp8, 2 * seed + 2, scale=scale)
    out = mx.gemm_bias_act(a.codes, a.scales, b.codes, b.scales, M, N, K, bias=bias, act=ACTS[act], residual=res, operands=FMT[fp8], **kw)
    mx.check_status()
    want = epilogue64(a.values, b.values, None if bias is None else f64(bias), act, None if res is None else f64(res))
    return out, want


SIZES = [(1, 8, 32), (1, 4128, 2080), (5, 136, 96), (128, 256, 256), (130, 264, 288), (257, 520, 1056), (300, 1032, 1280), (777, 96, 544)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_sizes(M, N, K, fp8, dtype):
    out, (z, ez, y, ey) = _run(M, N, K, fp8, "silu", _vector(N, F32, 1), _matrix(M, N, BF16, 2), dtype=dtype, want_z=True)
    assert out.y.dtype == dtype
    assert_output(out.y, y, ey, "y")
    assert_output(out.z, z, ez, "z")


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17])
@pytest.mark.parametrize("N,K", [(32, 32), (40, 96), (288, 4128), (4128, 160), (128, 2048)])
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
def test_few_rows(M, N, K, fp8):
    out, (z, ez, y, ey) = _run(M, N, K, fp8, "gelu_tanh", _vector(N, BF16, 1), _matrix(M, N, F32, 2, pad=8), dtype=F32, want_z=True, scale=-4)
    assert_output(out.y, y, ey, "y")
    assert_output(out.z, z, ez, "z")


def test_few_rows_keep_scales_at_the_ends_of_their_range():
    """2^(a - 127) 2^(b - 127) with each factor at an end of its range and the product inside fp32's; NaN scales in their row or column."""
    from tests.mx_testutil import tile_scales
    M, N, K = 4, 32, 64
    for fp8 in (False, True):
        a, b = Operand(M, K, fp8, 1), Operand(N, K, fp8, 2)
        ab, bb = np.array([[254, 0], [0, 254], [127, 127], [60, 194]], np.uint8), np.full((N, 2), 127, np.uint8)
        bb[:, 0], bb[:, 1] = 2, 250
        bb[8:], bb[20, 1] = 127, 255
        values = [v.values / np.repeat(np.exp2(v.byte - 127.0), 32, 1) for v in (a, b)]
        f = lambda x: np.repeat(np.exp2(x.astype(np.float64) - 127), 32, 1)  # noqa: E731
        y = mx.gemm_bias_act(a.codes, dev(tile_scales(ab, M, K)), b.codes, dev(tile_scales(bb, N, K)), M, N, K, dtype=F32, operands=FMT[fp8]).y
        ref = (values[0] * f(ab)) @ (values[1] * f(bb)).T
        size = np.abs(values[0] * f(ab)) @ np.abs(values[1] * f(bb)).T
        got = f64(y)
        assert np.isnan(got[:, 20]).all()
        ok = (size < 3e38) & (np.arange(N) != 20)
        assert ok.sum() == 8 + 23 + 23   # rows 0 (its first 8 columns), 2 and 3 (the others but the NaN's)
        assert_within(got[ok], ref[ok], 1e-5 * size[ok] + 2.0 ** -126, "values")


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias", [None, BF16, F32])
@pytest.mark.parametrize("res", [None, BF16, F32])
def test_epilogues(act, bias, res):
    M, N, K = 200, 328, 160
    out, (z, ez, y, ey) = _run(M, N, K, False, act, None if bias is None else _vector(N, bias, 3),
                               None if res is None else _matrix(M, N, res, 4, pad=24), dtype=F32, want_z=True, scale=-3)
    assert_output(out.y, y, ey, "y")
    assert_output(out.z, z, ez, "z")


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias", [None, BF16, F32])
@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_epilogues_of_four_lanes_a_row(act, bias, res, dtype):
    """A residual with N a multiple of 64: the other arrangement of the epilogue."""
    M, N, K = 200, 320, 160
    out, (z, ez, y, ey) = _run(M, N, K, False, act, None if bias is None else _vector(N, bias, 3), _matrix(M, N, res, 4, pad=24), dtype=dtype, want_z=True,
                               scale=-3)
    assert_output(out.y, y, ey, "y")
    assert_output(out.z, z, ez, "z")


@pytest.mark.parametrize("M,N,K", [(17, 64, 32), (300, 192, 96), (257, 320, 1056), (1000, 1088, 288)])
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
@pytest.mark.parametrize("fmt", [None, mx.FMT_MXFP4, mx.FMT_MXFP8], ids=["plain", "to mxfp4", "to mxfp8"])
def test_sizes_of_four_lanes_a_row(M, N, K, fp8, fmt):
    kw = dict(act="silu", bias=_vector(N, F32, 1), res=_matrix(M, N, BF16, 2))
    out, (z, ez, y, ey) = _run(M, N, K, fp8, dtype=F32, want_z=True, fmt=fmt, **kw)
    assert_output(out.y, y, ey, "y")
    assert_output(out.z, z, ez, "z")
    if fmt is not None:
        assert_encoding_of(out.codes, out.scales, out.y.cpu().numpy(), fmt == mx.FMT_MXFP8, "rows")
        alone = _run(M, N, K, fp8, want_y=False, fmt=fmt, **kw)[0]
        assert torch.equal(alone.codes, out.codes) and torch.equal(alone.scales, out.scales)


@pytest.mark.parametrize("M", [3, 16])
@pytest.mark.parametrize("fmt", [mx.FMT_MXFP4, mx.FMT_MXFP8], ids=["to mxfp4", "to mxfp8"])
def test_few_rows_encoded(M, fmt):
    N, K = 288, 224
    kw = dict(act="relu2", bias=_vector(N, F32, 1), res=_matrix(M, N, BF16, 2))
    out = _run(M, N, K, True, dtype=F32, fmt=fmt, **kw)[0]
    assert_encoding_of(out.codes, out.scales, out.y.cpu().numpy(), fmt == mx.FMT_MXFP8, "rows")


@pytest.mark.parametrize("N", [2048, 1892])
@pytest.mark.parametrize("K", [1024, 1312, 96])
def test_several_tiles_a_pair_have_the_plain_product_s_bits(N, K):
    """More tiles than CTA pairs, ragged at the end; the accumulator is that of mx.gemm."""
    N = N // 8 * 8
    M = 256 * ((torch.cuda.get_device_properties(0).multi_processor_count // 2 + 6 + 7) // 8) - 37
    a, b = Operand(M, K, False, 1), Operand(N, K, False, 2)
    args = (a.codes, a.scales, b.codes, b.scales, M, N, K)
    c = mx.gemm(*args)
    bias, res = _vector(N, F32, 1), _matrix(M, N, F32, 2)
    out = mx.gemm_bias_act(*args, bias=bias, residual=res, dtype=F32, want_z=True)
    mx.check_status()
    z = c + bias
    assert torch.equal(out.y, z + res) and torch.equal(out.z, z.bfloat16())


@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (130, 288, 96), (700, 1056, 320)])
@pytest.mark.parametrize("fmt", [mx.FMT_MXFP4, mx.FMT_MXFP8], ids=["to mxfp4", "to mxfp8"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_encoded_rows_are_the_encoding_of_y(M, N, K, fmt, dtype):
    kw = dict(act="gelu", bias=_vector(N, BF16, 5), res=_matrix(M, N, F32, 6))
    y32 = _run(M, N, K, False, dtype=F32, **kw)[0].y
    out = _run(M, N, K, False, dtype=dtype, fmt=fmt, **kw)[0]
    assert torch.equal(out.y, y32.to(dtype))
    assert_encoding_of(out.codes, out.scales, y32.cpu().numpy(), fmt == mx.FMT_MXFP8, "rows")
    alone = _run(M, N, K, False, want_y=False, fmt=fmt, **kw)[0]
    assert alone.y is None and torch.equal(alone.codes, out.codes) and torch.equal(alone.scales, out.scales)


@pytest.mark.parametrize("act", list(ACTS))
def test_activations_over_their_range(act):
    """A product of zeros leaves the bias: y = act(bias), tails and ends of fp32's range among it."""
    x = np.concatenate([np.linspace(-110, 110, 2201), np.linspace(-6, 6, 2401), [0.0, -0.0, 1e-30, -1e-30, 1e18, -1e18, 3e4, -3e4]])
    x = np.resize(x, (x.size + 7) // 8 * 8).astype(np.float32)
    N = x.size
    a, b = Operand(3, 32, False, 1, lines_zero=slice(None)), Operand(N, 32, False, 2)
    out = mx.gemm_bias_act(a.codes, a.scales, b.codes, b.scales, 3, N, 32, bias=dev(x), act=ACTS[act], dtype=F32)
    x = x.astype(np.float64)
    ref = np.minimum(act64(act, x), np.float64(np.finfo(np.float32).max)) if act == "relu2" else act64(act, x)
    ok = np.isfinite(act64(act, x).astype(np.float32))
    assert_within(f64(out.y)[:, ok], np.broadcast_to(ref, (3, N))[:, ok], (act_bound(act, x) + 2.0 ** -126 * (np.abs(ref) < 2.0 ** -120))[ok], act)


@pytest.mark.parametrize("act", list(ACTS))
def test_infinities_and_nan_give_what_the_formula_gives(act):
    x = torch.tensor([float("inf"), float("-inf"), float("nan"), 1.0] * 2, dtype=F32)
    a, b = Operand(2, 32, False, 1, lines_zero=slice(None)), Operand(8, 32, False, 2)
    y = mx.gemm_bias_act(a.codes, a.scales, b.codes, b.scales, 2, 8, 32, bias=x.cuda(), act=ACTS[act], dtype=F32).y.cpu()
    low = {"none": float("-inf"), "relu": 0.0, "relu2": 0.0}.get(act, float("nan"))
    for row in y:
        assert row[0] == float("inf") and torch.isnan(row[2])
        assert torch.isnan(row[1]) if low != low else row[1] == low


def test_a_nan_scale_stays_in_its_row_or_column():
    M, N, K = 300, 320, 288
    a, b = Operand(M, K, False, 1), Operand(N, K, False, 2)
    clean = mx.gemm_bias_act(a.codes, a.scales, b.codes, b.scales, M, N, K, dtype=F32).y
    from tests.mx_testutil import tile_scales
    a.byte[131, 8], b.byte[257, 0] = 0xFF, 0xFF
    y = mx.gemm_bias_act(a.codes, dev(tile_scales(a.byte, M, K)), b.codes, dev(tile_scales(b.byte, N, K)), M, N, K, dtype=F32, fmt=mx.FMT_MXFP8)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[131], bad[:, 257] = True, True
    assert torch.equal(torch.isnan(y.y), bad) and torch.equal(y.y[~bad], clean[~bad])
    from tests.mx_testutil import untile_scales
    s = untile_scales(y.scales.cpu().numpy(), M, N)
    assert (s[131] == 0xFF).all() and (s[:, 8] == 0xFF).all() and (np.delete(np.delete(s, 131, 0), 8, 1) != 0xFF).all()


def test_the_residual_updated_in_place():
    M, N, K = 513, 264, 96
    for dtype in (BF16, F32):
        res = _matrix(M, N, dtype, 7).contiguous()
        want = _run(M, N, K, False, "relu", res=res.clone(), dtype=dtype)[0].y
        out, _ = _run(M, N, K, False, "relu", res=res, out=res)
        assert out.y is res and torch.equal(res, want)


def test_no_contraction_and_no_rows():
    bias, res = _vector(40, F32, 1), _matrix(7, 40, BF16, 2)
    out, (z, ez, y, ey) = _run(7, 40, 0, False, "gelu_tanh", bias, res, dtype=F32, want_z=True)
    assert_output(out.y, y, ey, "y")
    assert_output(out.z, z, ez, "z")
    for M, N in ((0, 64), (64, 0)):
        out = _run(M, N, 64, False, "relu")[0]
        assert out.y.shape == (M, N)


def test_bf16_rows_off_a_32_byte_boundary():
    M, N, K = 140, 264, 96   # 528 bytes a row
    want = _run(M, N, K, False, "gelu", dtype=BF16)[0].y
    flat = torch.zeros(M * N + 8, dtype=BF16, device="cuda")
    out = flat[8:].view(M, N)
    _run(M, N, K, False, "gelu", out=out)
    assert torch.equal(out, want) and not flat[:8].any()


def test_outputs_beyond_32_bits_of_bytes():
    M, N, K = 66000, 16384, 32
    a, b = Operand(M, K, False, 1), Operand(N, K, False, 2)
    y = mx.gemm_bias_act(a.codes, a.scales, b.codes, b.scales, M, N, K, dtype=F32).y
    mx.check_status()
    rows = [0, 255, 32767, 65535, 65536, 65999]
    ref = a.values[rows] @ b.values.T
    assert_within(y[rows], ref, 1e-5 * (np.abs(a.values[rows]) @ np.abs(b.values).T), "rows")


def test_another_stream_and_a_captured_graph():
    M, N, K = 384, 512, 256
    a, b = Operand(M, K, False, 1), Operand(N, K, False, 2)
    args = (a.codes, a.scales, b.codes, b.scales, M, N, K)
    bias = _vector(N, F32, 1)
    call = lambda **kw: mx.gemm_bias_act(*args, bias=bias, act=mx.ACT_SILU, want_z=True, fmt=mx.FMT_MXFP4, **kw)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    grad = mx.bias_act_backward(want.y, want.z, mx.ACT_SILU, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    eager = mx.bias_act_backward(want.y, want.z, mx.ACT_SILU)
    for p, q in zip((*got, grad.dz, grad.dbias), (*want, eager.dz, eager.dbias)):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
        back = mx.bias_act_backward(held.y, held.z, mx.ACT_SILU)
    for t in (*held, back.dz, back.dbias):
        t.zero_()
    graph.replay()
    for p, q in zip((*held, back.dz, back.dbias), (*want, eager.dz, eager.dbias)):
        assert torch.equal(p, q)
    bias.mul_(2)
    graph.replay()
    assert torch.equal(held.y, call().y)


# ---------------------------------------------------------------------------- the gradient
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dy_type", [BF16, F32])
@pytest.mark.parametrize("z_type", [BF16, F32])
@pytest.mark.parametrize("T,N", [(1, 8), (97, 2080), (129, 264), (1000, 520)])
def test_gradient(act, dy_type, z_type, T, N):
    dy, z = _matrix(T, N, dy_type, 1, pad=16), _matrix(T, N, z_type, 2, pad=8, spread=3.0)
    out = mx.bias_act_backward(dy, z, ACTS[act])
    d, x = f64(dy), f64(z)
    slope = slope64(act, x)
    ref = d * slope
    # The slope's terms are each within (16 + 4 x^2) u of themselves; they may cancel, so their sizes count, and the product rounds.
    parts = np.abs(slope) if act in ("none", "relu", "relu2") else 1.0 + np.abs(x) * np.exp(-np.minimum(np.abs(x), 30) / 2) * (1 + x * x)
    err = np.abs(d) * (20 + 4 * np.minimum(x * x, 100)) * U * parts + 2.0 ** -126
    assert_within(out.dz, ref, err + UB * (np.abs(ref) + err), "dz")
    # A column's sum: terms a lane adds (T / 8 at most), 16 warps or 128 shares: log-like parts, each rounding of a partial sum.
    total = (np.minimum(T, 256) / 8 + 16 + 24) * U * np.abs(ref).sum(0) + err.sum(0)
    assert_within(out.dbias, ref.sum(0), total, "dbias")
    again = mx.bias_act_backward(dy, z, ACTS[act])
    assert torch.equal(again.dbias, out.dbias) and torch.equal(again.dz, out.dz)


@pytest.mark.parametrize("act", [n for n in ACTS if n not in ("none", "relu")])
def test_slopes_are_the_activations_differences(act):
    """The kernel's slope against central differences of its own activation's 64-bit form."""
    x = np.linspace(-9, 9, 1440)
    z = dev(x.astype(np.float32)[None])
    got = f64(mx.bias_act_backward(torch.ones_like(z), z, ACTS[act], want_dz=False).dbias)
    x, h = f64(z)[0], 1e-4
    differences = (act64(act, x + h) - act64(act, x - h)) / (2 * h)
    # h^2 / 6 of a third derivative below 3, the difference's 64-bit roundings, and the kernel's own error
    assert np.abs(got - differences).max() < 0.5 * h * h * (6 if act == "relu2" else 1) + 1e-11 * 100 + 2e-6 + (2 * h if act == "relu2" else 0)


@pytest.mark.parametrize("fmt", [mx.FMT_MXFP4, mx.FMT_MXFP8])
@pytest.mark.parametrize("T,N", [(1, 32), (130, 288), (515, 1056)])
def test_gradient_encoded(fmt, T, N):
    dy, z = _matrix(T, N, F32, 1), _matrix(T, N, BF16, 2)
    out = mx.bias_act_backward(dy, z, mx.ACT_RELU2, fmt=fmt, want_dbias=False)
    assert out.dbias is None
    dz = (dy * (2 * z.float().clamp(min=0))).cpu().numpy()  # the same two fp32 products
    assert torch.equal(out.dz, dev(dz).bfloat16())
    assert_encoding_of(out.codes, out.scales, dz, fmt == mx.FMT_MXFP8, "dz")


def test_bias_gradient_alone_and_empty_calls():
    dy = _matrix(3000, 264, BF16, 1)
    out = mx.bias_act_backward(dy, want_dz=False)
    assert out.dz is None
    assert_within(out.dbias, f64(dy).sum(0), 80 * U * np.abs(f64(dy)).sum(0), "dbias")
    assert torch.equal(mx.bias_act_backward(dy[:0], want_dz=False).dbias, torch.zeros(264, device="cuda"))
    assert mx.bias_act_backward(dy[:, :0]).dz.shape == (3000, 0)


def test_gradient_of_many_rows_uses_bounded_workspace():
    T, N = 70001, 64
    dy = torch.ones(T, N, dtype=BF16, device="cuda")
    out = mx.bias_act_backward(dy, want_dz=False, ws=torch.empty(mx.bias_act_backward_workspace_bytes(T, N), dtype=torch.uint8, device="cuda"))
    assert mx.bias_act_backward_workspace_bytes(T, N) <= 128 * N * 4
    assert (out.dbias == T).all()


def test_few_rows_whose_scales_pass_32_bits():
    N, K = 8, 2 ** 29 + 4096     # a line's scales end 2^31 + 16384 bytes behind its first
    blocks, value = K // 32, {}
    operands = []
    for lines in (1, N):
        codes, scales = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (lines * K // 2, mx.lib().mx_scales_bytes(lines, K)))
        for line in range(lines):
            for at, b in enumerate((0, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 5, blocks - 1)):
                first = line * K // 2 + b * 16
                codes[first:first + 16] = 0x22   # ones
                scales[(b >> 2) * 512 + line * 16 + (b & 3)] = 127 + at + (lines > 1) * line
                value[lines, line, at] = 2.0 ** (at + (lines > 1) * line)
        operands += [codes, scales]
    y = mx.gemm_bias_act(*operands, 1, N, K, dtype=F32).y
    mx.check_status()
    assert y.tolist() == [[32 * sum(value[1, 0, at] * value[N, line, at] for at in range(5)) for line in range(N)]]
