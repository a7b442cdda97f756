"""Plans, rows in and out, and products grouped by expert against 64-bit
forms; tolerances in product_testutil."""
import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.mx_testutil import GEMM_TOL, tile_scales
from tests.product_testutil import (ACTS, U, UB, Operand, assert_encoding_of, assert_output, assert_within, dev, device_plan, epilogue64,
                                    f64, plan64, routing)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FMT = {False: mx.FMT_MXFP4, True: mx.FMT_MXFP8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


# ---------------------------------------------------------------------------- plan
@pytest.mark.parametrize("T,picks,E,drop,skew", [(1, 1, 1, 0, 0), (9, 4, 16, 0, 1), (300, 2, 64, 0.1, 2), (1024, 2, 8, 0, 0), (1025, 2, 8, 0, 0),
                                                 (5000, 8, 512, 0.05, 0.5), (40000, 1, 3, 0, 3), (70000, 4, 33, 0.5, 1), (64, 3, 5, 1.0, 0)])
@pytest.mark.parametrize("wide", [False, True], ids=["int32", "int64"])
def test_plan(T, picks, E, drop, skew, wide):
    index = routing(T, picks, E, T + E, drop, skew)
    plan = mx.expert_plan(dev(index.astype(np.int64) if wide else index), E)
    for got, want, name in zip(plan, plan64(index, E), mx.ExpertPlan._fields):
        assert np.array_equal(got.cpu().numpy(), want), name


def test_plan_of_one_expert_twice_and_of_numbers_that_name_none():
    index = np.array([[2, 2], [7, -5], [2, 0], [2 ** 31 - 1, -2 ** 31]], np.int32)
    plan = mx.expert_plan(dev(index), 3)
    want = plan64(np.where((index >= 0) & (index < 3), index, -1).astype(np.int32), 3)
    for got, ref in zip(plan, want):
        assert np.array_equal(got.cpu().numpy(), ref)
    far = mx.expert_plan(dev(np.array([[2 ** 32 + 1, 1]], np.int64)), 3)
    assert far.slot.tolist() == [[-1, 0]]


def test_plan_of_no_tokens():
    plan = mx.expert_plan(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 5)
    assert plan.offsets.tolist() == [0] * 6 and plan.counts.tolist() == [0] * 5 and plan.source.numel() == 0
    assert mx.expert_dispatch(torch.empty(0, 64, device="cuda"), plan).y.shape == (0, 64)
    res = torch.ones(0, 64, device="cuda")
    assert mx.expert_combine(torch.empty(0, 64, device="cuda"), plan, residual=res).shape == (0, 64)


# ---------------------------------------------------------------------------- rows in and out
SHAPES = [(1, 1, 1, 8, 0), (9, 4, 16, 2080, 0), (37, 8, 64, 1056, 0.2), (300, 3, 7, 320, 0.1), (129, 2, 4, 4096, 0), (20, 2, 3, 64, 1.0)]


@pytest.mark.parametrize("T,picks,E,K,drop", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", [None, mx.FMT_MXFP4, mx.FMT_MXFP8])
def test_dispatch(T, picks, E, K, drop, dtype, fmt):
    if fmt is not None:
        K = -(-K // 32) * 32
    plan, (offsets, counts, slot, source) = device_plan(routing(T, picks, E, 1, drop), E)
    x = (torch.randn(T, K + 24, generator=torch.Generator().manual_seed(1)) * 3).to(dtype).cuda()[:, :K]
    out = mx.expert_dispatch(x, plan, fmt=fmt)
    rows = np.zeros((source.size, K), np.float32)
    rows[source >= 0] = x.float().cpu().numpy()[source[source >= 0] // picks]
    assert torch.equal(out.y, dev(rows).bfloat16())
    if fmt is not None:
        assert_encoding_of(out.codes, out.scales, rows, fmt == mx.FMT_MXFP8, "rows")
        alone = mx.expert_dispatch(x, plan, fmt=fmt, want_y=False)
        assert alone.y is None and torch.equal(alone.codes, out.codes) and torch.equal(alone.scales, out.scales)


@pytest.mark.parametrize("T,picks,E,K,drop", SHAPES)
@pytest.mark.parametrize("row,res", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32), (BF16, None), (F32, None)])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(T, picks, E, K, drop, row, res, weighted):
    plan, (_, _, slot, source) = device_plan(routing(T, picks, E, 2, drop), E)
    g = torch.Generator().manual_seed(2)
    rows = torch.randn(source.size, K + 8, generator=g).to(row).cuda()[:, :K]
    w = torch.rand(T, picks, generator=g).cuda()
    r = None if res is None else torch.randn(T, K + 16, generator=g).to(res).cuda()[:, :K]
    y = mx.expert_combine(rows, plan, weights=w if weighted else None, residual=r)
    assert y.dtype == (row if res is None else res)
    there = slot >= 0
    weight = np.where(there, f64(w) if weighted else 1.0, 0.0)[:, :, None]
    terms = weight * f64(rows)[np.where(there, slot, 0)]
    ref = terms.sum(1) + (0 if r is None else f64(r))
    err = (picks + 1) * U * (np.abs(terms).sum(1) + (0 if r is None else np.abs(f64(r))))
    assert_output(y, ref, err, "y")


def test_combine_into_the_residual_and_with_dropped_nan_rows():
    T, picks, E, K = 50, 2, 4, 264
    plan, (_, counts, slot, source) = device_plan(routing(T, picks, E, 3, 0.3), E)
    rows = torch.randn(source.size, K, device="cuda")
    rows[torch.from_numpy(source < 0).cuda()] = float("nan")  # rows without a token are not read
    w = torch.rand(T, picks, device="cuda")
    w[torch.from_numpy(slot < 0).cuda()] = float("nan")
    res = torch.randn(T, K, device="cuda").bfloat16()
    want = mx.expert_combine(rows, plan, w, res.clone())
    assert torch.isfinite(want).all()
    assert mx.expert_combine(rows, plan, w, res, out=res) is res and torch.equal(res, want)
    assert mx.expert_combine(rows, plan, w, res, dtype=F32).dtype == F32


@pytest.mark.parametrize("T,picks,E,K,drop", SHAPES)
@pytest.mark.parametrize("dy_type", [BF16, F32])
@pytest.mark.parametrize("row", [BF16, F32])
def test_combine_gradient(T, picks, E, K, drop, dy_type, row):
    plan, (_, _, slot, source) = device_plan(routing(T, picks, E, 4, drop), E)
    g = torch.Generator().manual_seed(4)
    rows, w = torch.randn(source.size, K, generator=g).to(row).cuda(), torch.rand(T, picks, generator=g).cuda()
    dy = torch.randn(T, K + 8, generator=g).to(dy_type).cuda()[:, :K]
    fmt = mx.FMT_MXFP4 if K % 32 == 0 else None
    out = mx.expert_combine_backward(dy, rows, plan, w, fmt=fmt)
    real = source >= 0
    grad = np.zeros((source.size, K), np.float32)
    grad[real] = (w.flatten()[dev(source[real]).long()][:, None] * dy.float()[dev(source[real] // picks).long()]).cpu().numpy()
    assert torch.equal(out.y, dev(grad).bfloat16())
    if fmt:
        assert_encoding_of(out.codes, out.scales, grad, False, "rows' gradient")
    there = slot >= 0
    terms = f64(dy)[:, None] * f64(rows)[np.where(there, slot, 0)] * there[:, :, None]
    # a lane's chunks, eight warps, a tree over the lanes
    err = (K / 256 / 8 * 4 + 8 + 8 + 5) * U * np.abs(terms).sum(2) + 1e-30
    assert_within(out.dweights, terms.sum(2), err, "dweights")
    assert torch.equal(out.dweights, mx.expert_combine_backward(dy, rows, plan, w, want_y=False).dweights)
    assert mx.expert_combine_backward(dy, None, plan, w, want_dweights=False).dweights is None


def test_dispatch_and_combine_are_each_other_s_gradients():
    """<dispatch(x), g> = <x, combine(g)>, and the weights' gradient against differences, in whole numbers."""
    T, picks, E, K = 40, 3, 6, 64
    plan, _ = device_plan(routing(T, picks, E, 5, 0.2), E)
    x = torch.randint(-8, 9, (T, K), device="cuda").float()
    g = torch.randint(-8, 9, (plan.source.numel(), K), device="cuda").float()
    assert (mx.expert_dispatch(x, plan).y.double() * g.double()).sum() == (x.double() * mx.expert_combine(g, plan).double()).sum()
    w = torch.randint(-4, 5, (T, picks), device="cuda").float()
    dw = mx.expert_combine_backward(x, g, plan, w).dweights
    base = (mx.expert_combine(g, plan, w).double() * x.double()).sum(1)
    for j in range(picks):
        step = w.clone()
        step[:, j] += 1
        assert torch.equal((mx.expert_combine(g, plan, step).double() * x.double()).sum(1) - base, dw[:, j].double())


# ---------------------------------------------------------------------------- products along the rows
def _experts_operand(E, N, K, fp8, seed, scale=-2):
    parts = [Operand(N, K, fp8, seed + 10 * e, scale=scale) for e in range(E)]
    return torch.cat([p.codes for p in parts]), torch.cat([p.scales for p in parts]), [p.values for p in parts]


def _rows_case(T, picks, E, N, K, fp8, drop=0.0, skew=0.5, seed=0, scale=-2):
    index = routing(T, picks, E, seed, drop, skew)
    plan, parts = device_plan(index, E)
    a = Operand(parts[3].size, K, fp8, seed + 1, scale=scale, lines_zero=parts[3] < 0)
    b_codes, b_scales, b_values = _experts_operand(E, N, K, fp8, seed + 2, scale)
    return plan, parts, a, b_codes, b_scales, b_values


@pytest.mark.parametrize("T,picks,E,N,K,drop,skew", [(1, 1, 1, 8, 32, 0, 0), (12, 2, 64, 264, 96, 0, 0.5), (300, 2, 5, 520, 288, 0.1, 1), (700, 3, 6, 256, 1056, 0, 2),
                                                      (1500, 2, 3, 1032, 544, 0, 0), (40, 8, 512, 64, 64, 0, 0), (600, 1, 4, 136, 128, 0.5, 4), (30, 2, 4, 64, 64, 1.0, 0),
                                                      (3, 2, 8, 520, 96, 0, 0), (16, 1, 30, 264, 2080, 0.1, 6), (5, 4, 512, 40, 4128, 0, 1)])
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
def test_rows(T, picks, E, N, K, drop, skew, fp8):
    plan, (offsets, counts, slot, source), a, bc, bs, bv = _rows_case(T, picks, E, N, K, fp8, drop, skew, seed=T)
    bias = torch.randn(E, N, generator=torch.Generator().manual_seed(1)).cuda()
    out = mx.gemm_experts(a.codes, a.scales, bc, bs, plan, N, K, bias=bias, act=mx.ACT_GELU, dtype=F32, want_z=True, operands=FMT[fp8])
    mx.check_status()
    P = source.size
    z, ez, y, ey = (np.zeros((P, N)) for _ in range(4))
    for e in range(E):
        r = slice(offsets[e], offsets[e] + counts[e])
        if counts[e]:
            z[r], ez[r], y[r], ey[r] = epilogue64(a.values[r], bv[e], f64(bias[e]), "gelu", None)
    assert_output(out.y, y, ey, "y")
    assert_output(out.z, z, ez, "z")


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias", [None, BF16, F32])
def test_rows_epilogues(act, bias):
    T, picks, E, N, K = 260, 2, 3, 96, 64
    plan, (offsets, counts, _, source), a, bc, bs, bv = _rows_case(T, picks, E, N, K, False, 0.1, seed=3, scale=-3)
    b = None if bias is None else torch.randn(E, N, generator=torch.Generator().manual_seed(2)).to(bias).cuda()
    out = mx.gemm_experts(a.codes, a.scales, bc, bs, plan, N, K, bias=b, act=ACTS[act])
    y, ey = np.zeros((source.size, N)), np.zeros((source.size, N))
    for e in range(E):
        r = slice(offsets[e], offsets[e] + counts[e])
        _, _, y[r], ey[r] = epilogue64(a.values[r], bv[e], None if b is None else f64(b[e]), act, None)
    assert_output(out.y, y, ey, "y")


@pytest.mark.parametrize("fmt", [mx.FMT_MXFP4, mx.FMT_MXFP8])
def test_rows_encoded(fmt):
    T, picks, E, N, K = 333, 2, 9, 288, 96
    plan, parts, a, bc, bs, _ = _rows_case(T, picks, E, N, K, False, 0.2, 2.0, seed=5)
    args = (a.codes, a.scales, bc, bs, plan, N, K)
    bias = torch.randn(E, N, generator=torch.Generator().manual_seed(3)).cuda()
    y = mx.gemm_experts(*args, bias=bias, act=mx.ACT_SILU, dtype=F32).y
    out = mx.gemm_experts(*args, bias=bias, act=mx.ACT_SILU, want_y=False, fmt=fmt)
    assert_encoding_of(out.codes, out.scales, y.cpu().numpy(), fmt == mx.FMT_MXFP8, "rows")


@pytest.mark.parametrize("fmt", [mx.FMT_MXFP4, mx.FMT_MXFP8])
def test_few_rows_encoded(fmt):
    T, picks, E, N, K = 4, 2, 20, 288, 96
    plan, parts, a, bc, bs, _ = _rows_case(T, picks, E, N, K, False, 0.2, 2.0, seed=7)
    args = (a.codes, a.scales, bc, bs, plan, N, K)
    out = mx.gemm_experts(*args, act=mx.ACT_GELU_TANH, dtype=F32, fmt=fmt)
    assert_encoding_of(out.codes, out.scales, out.y.cpu().numpy(), fmt == mx.FMT_MXFP8, "rows")


def test_rows_of_experts_hold_what_separate_products_hold():
    """Several tiles a pair, bit for bit the dense product of each expert."""
    T, picks, E, N, K = 6000, 2, 7, 1032, 640
    plan, (offsets, counts, _, source), a, bc, bs, _ = _rows_case(T, picks, E, N, K, False, 0.0, 1.0, seed=6)
    y = mx.gemm_experts(a.codes, a.scales, bc, bs, plan, N, K, dtype=F32).y
    mx.check_status()
    want = torch.zeros_like(y)
    n = mx.scales_bytes(N, K)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            per = mx.scales_bytes(128, K)
            want[lo:hi] = mx.gemm(a.codes[lo:hi].contiguous(), a.scales[lo // 128 * per:hi // 128 * per].contiguous(), bc[e * N:(e + 1) * N].contiguous(),
                                  bs[e * n:(e + 1) * n].contiguous(), hi - lo, N, K)
    assert torch.equal(y, want)


# ---------------------------------------------------------------------------- products along the contraction
@pytest.mark.parametrize("T,picks,E,M,N,drop,skew", [(1, 1, 1, 8, 8, 0, 0), (301, 2, 16, 136, 264, 0.1, 2), (700, 3, 6, 328, 96, 0, 1), (2000, 1, 3, 520, 1032, 0, 0),
                                                      (20, 2, 300, 64, 72, 0, 0), (30, 2, 4, 64, 64, 1.0, 0), (1800, 2, 5, 1300, 256, 0, 1)])
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_depth(T, picks, E, M, N, drop, skew, fp8, dtype):
    plan, (offsets, counts, _, source) = device_plan(routing(T, picks, E, T, drop, skew), E)
    P = source.size
    a, b = Operand(M, P, fp8, 1), Operand(N, P, fp8, 2)   # no zeros in the padding: the slices' ends count
    c = mx.gemm_experts_wgrad(a.codes, a.scales, b.codes, b.scales, plan, M, N, dtype=dtype, operands=FMT[fp8])
    mx.check_status()
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        ref, size = a.values[:, s] @ b.values[:, s].T, np.abs(a.values[:, s]) @ np.abs(b.values[:, s]).T
        assert_output(c[e], ref, GEMM_TOL * size, f"expert {e}")


@pytest.mark.parametrize("rot,block", [(mx.ROT_NONE, 32), (mx.ROT_HADAMARD_DET, 32), (mx.ROT_HADAMARD_DET, 128), (mx.ROT_HADAMARD_RAND, 64)])
def test_linear_wgrad_is_the_dense_wgrad_of_each_expert(rot, block):
    T, picks, E, N, K = 500, 2, 4, 264, 136
    index = routing(T, picks, E, 8)
    plan = mx.expert_plan(dev(index), E)
    g = torch.Generator().manual_seed(8)
    dy, x = (mx.expert_dispatch(torch.randn(T, n, generator=g).cuda(), plan).y for n in (N, K))
    dw = mx.linear_experts_wgrad(dy, x, plan, rot=rot, rot_block=block, seed=5)
    mx.check_status()
    off = plan.offsets.tolist()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if rot != mx.ROT_HADAMARD_RAND:   # the signs go by the row's place in the call
            assert torch.equal(dw[e], mx.linear_wgrad(dy[lo:hi].contiguous(), x[lo:hi].contiguous(), rot=rot, rot_block=block))
        true = dy[lo:hi].double().T @ x[lo:hi].double()
        assert (dw[e].double() - true).norm() < 0.25 * true.norm()


def test_linear_wgrad_in_mxfp8_and_its_refusals():
    T, picks, E, N, K = 300, 2, 3, 64, 96
    plan = mx.expert_plan(dev(routing(T, picks, E, 9)), E)
    g = torch.Generator().manual_seed(9)
    dy, x = (mx.expert_dispatch(torch.randn(T, n, generator=g).cuda(), plan).y for n in (N, K))
    dw = mx.linear_experts_wgrad(dy, x, plan, operands=mx.FMT_MXFP8, rot=mx.ROT_NONE)
    off = plan.offsets.tolist()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        assert torch.equal(dw[e], mx.linear_wgrad_mxfp8(dy[lo:hi].contiguous(), x[lo:hi].contiguous()))
    for kw in (dict(operands=mx.FMT_MXFP8), dict(rot_block=256), dict(operands=mx.FMT_MXFP8, rot=mx.ROT_NONE, rnd=mx.ROUND_SR)):
        with pytest.raises(mx.MXError):
            mx.linear_experts_wgrad(dy, x, plan, **kw)


@pytest.mark.parametrize("rows,cols,contract", [(128, 96, mx.CONTRACT_COLS), (136, 96, mx.CONTRACT_COLS), (96, 136, mx.CONTRACT_ROWS), (256, 64, mx.CONTRACT_ROWS)])
def test_quantize_experts(rows, cols, contract):
    w = torch.randn(5, rows, cols, device="cuda").bfloat16()
    codes, scales = mx.quantize_experts(w, contract)
    one = [mx.quantize(w[e].contiguous(), contract) for e in range(5)]
    assert torch.equal(codes, torch.cat([c for c, _ in one])) and torch.equal(scales, torch.cat([s for _, s in one]))
    if contract == mx.CONTRACT_ROWS:
        codes, scales = mx.quantize_experts(w, contract, operands=mx.FMT_MXFP8)
        one = [mx.quantize_mxfp8(w[e].contiguous()) for e in range(5)]
        assert torch.equal(codes, torch.cat([c for c, _ in one])) and torch.equal(scales, torch.cat([s for _, s in one]))
    else:
        with pytest.raises(mx.MXError):
            mx.quantize_experts(w, contract, operands=mx.FMT_MXFP8)


# ---------------------------------------------------------------------------- together
def _layer(x, index, w, w1, w2, d_out, E, F):
    """One layer of experts, forward and backward, all on the device."""
    K = x.shape[1]
    plan = mx.expert_plan(index, E)
    rows = mx.expert_dispatch(x, plan, fmt=mx.FMT_MXFP4)
    h = mx.gemm_experts(rows.codes, rows.scales, *mx.quantize_experts(w1), plan, F, K, act=mx.ACT_SILU, want_z=True, fmt=mx.FMT_MXFP4)
    out = mx.gemm_experts(h.codes, h.scales, *mx.quantize_experts(w2), plan, K, F)
    y = mx.expert_combine(out.y, plan, w, x)
    g = mx.expert_combine_backward(d_out, out.y, plan, w, fmt=mx.FMT_MXFP4)
    dh = mx.gemm_experts(g.codes, g.scales, *mx.quantize_experts(w2, mx.CONTRACT_ROWS), plan, F, K)
    dw2 = mx.linear_experts_wgrad(g.y, h.y, plan)
    dz = mx.bias_act_backward(dh.y, h.z, mx.ACT_SILU, want_dbias=False, fmt=mx.FMT_MXFP4)
    dx = mx.gemm_experts(dz.codes, dz.scales, *mx.quantize_experts(w1, mx.CONTRACT_ROWS), plan, K, F)
    dw1 = mx.linear_experts_wgrad(dz.dz, rows.y, plan)
    return y, mx.expert_combine(dx.y, plan, residual=d_out), dw1, dw2, g.dweights


def test_a_layer_of_experts_forward_backward_and_captured():
    T, picks, E, K, F = 200, 2, 6, 128, 256
    g = torch.Generator().manual_seed(11)
    x, d_out = (torch.randn(T, K, generator=g).cuda().bfloat16() for _ in range(2))
    index = dev(routing(T, picks, E, 11))
    w = torch.rand(T, picks, generator=g).cuda()
    w1, w2 = ((torch.randn(E, *s, generator=g) * s[1] ** -0.5).cuda().bfloat16() for s in ((F, K), (K, F)))
    eager = _layer(x, index, w, w1, w2, d_out, E, F)
    mx.check_status()
    # The layer in 64 bits, without quantisation: its gradients by autograd.
    leaves = [t.double().requires_grad_() for t in (x, w1, w2, w)]
    X, W1, W2, R = leaves
    y = X
    for j in range(picks):
        e = index[:, j].long()
        h = torch.nn.functional.silu(torch.einsum("tk,tfk->tf", X, W1[e]))
        y = y + R[:, j:j + 1] * torch.einsum("tf,tkf->tk", h, W2[e])
    true = torch.autograd.grad(y, leaves, d_out.double())
    # FP4 operands: an element is off by 2^-3 to 2^-2 of itself, about 0.12 in the mean square of a product of two, and twice that through two products.
    for got, ref, name in ((eager[0], y, "y"), (eager[1], true[0], "dx"), (eager[2], true[1], "dw1"), (eager[3], true[2], "dw2"), (eager[4], true[3], "dweights")):
        off = ((got.double() - ref).norm() / ref.norm()).item()
        assert off < 0.45, (name, off)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _layer(x, index, w, w1, w2, d_out, E, F)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        held = _layer(x, index, w, w1, w2, d_out, E, F)
    graph.replay()
    for p, q in zip(held, eager):
        assert torch.equal(p, q)
    index.copy_(dev(routing(T, picks, E, 12, 0.2, 2.0)))   # another routing in the same graph
    graph.replay()
    for p, q in zip(held, _layer(x, index, w, w1, w2, d_out, E, F)):
        assert torch.equal(p, q)


def test_calls_at_once_on_two_streams_hold_what_calls_in_turn_hold():
    # A layer's forward and weight gradients on each stream, with plans of their own.
    E, N, K, picks = 6, 520, 288, 2

    def call(seed):
        x = torch.randn(900 + 100 * seed, K, generator=torch.Generator().manual_seed(seed)).cuda()
        index = dev(routing(x.shape[0], picks, E, seed, 0.1, 1))
        w, wt = _experts_operand(E, N, K, False, seed)[:2], torch.rand(x.shape[0], picks, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        torch.cuda.synchronize()

        def run():
            plan = mx.expert_plan(index, E)
            rows = mx.expert_dispatch(x, plan, fmt=mx.FMT_MXFP4)
            o = mx.gemm_experts(rows.codes, rows.scales, *w, plan, N, K, act=mx.ACT_SILU, want_z=True)
            y = mx.expert_combine(o.y, plan, wt)
            g = mx.expert_combine_backward(y, o.y, plan, wt)
            b = mx.bias_act_backward(g.y, o.z, mx.ACT_SILU)
            return [*plan, rows.y, o.y, y, g.dweights, b.dz, b.dbias, mx.linear_experts_wgrad(b.dz, rows.y, plan)]
        return run
    calls = [call(1), call(2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = []
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(c())
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(u, v))
    mx.check_status()


def test_a_plan_s_parts_are_tensors_of_their_own():
    index = dev(routing(37, 3, 5, 1, 0.1))
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            plan, want = mx.expert_plan(index, 5), plan64(index.cpu().numpy(), 5)
            for i, part in enumerate(plan):
                assert part.is_contiguous() and part.data_ptr() % 16 == 0
                part.fill_(7)
                for other, w in list(zip(plan, want))[i + 1:]:
                    assert np.array_equal(other.cpu().numpy(), w)
    source = mx.expert_plan(index, 5).source
    torch.empty(1 << 20, device="cuda").fill_(1)   # what the other parts took is not given away while one is in use
    assert np.array_equal(source.cpu().numpy(), want[3])
    assert mx.expert_plan(index[:0], 5).source.shape == (0,)


# Blocks of 128 columns: more than 32 tiles of 256 columns, and no more than 128 rows an expert.
@pytest.mark.parametrize("T,picks,E,N,K,skew", [(33, 1, 64, 8, 32, 0), (150, 1, 64, 264, 416, 20), (150, 1, 64, 520, 1056, 4), (9, 4, 40, 1032, 96, 1),
                                                (20, 3, 512, 136, 2080, 0), (60, 2, 512, 72, 4128, 3), (40, 1, 64, 264, 0, 1)])
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
def test_many_experts_of_few_rows(T, picks, E, N, K, skew, fp8):
    plan, (offsets, counts, slot, source), a, bc, bs, bv = _rows_case(T, picks, E, N, K, fp8, 0.1, skew, seed=T)
    assert source.size <= 128 * E and source.size // 128 * -(-N // 256) > 32
    bias = torch.randn(E, N, generator=torch.Generator().manual_seed(1)).cuda()
    want = [np.zeros((source.size, N)) for _ in range(4)]
    for e in np.flatnonzero(counts):
        r = slice(offsets[e], offsets[e] + counts[e])
        for w, v in zip(want, epilogue64(a.values[r], bv[e], f64(bias[e]), "silu", None)):
            w[r] = v
    for dtype in (F32, BF16):
        out = mx.gemm_experts(a.codes, a.scales, bc, bs, plan, N, K, bias=bias, act=mx.ACT_SILU, dtype=dtype, want_z=True, operands=FMT[fp8])
        mx.check_status()
        assert_output(out.y, want[2], want[3], "y")
        assert_output(out.z, want[0], want[1], "z")


@pytest.mark.parametrize("fmt", [mx.FMT_MXFP4, mx.FMT_MXFP8])
@pytest.mark.parametrize("T,skew", [(20, 0), (150, 20)])
def test_many_experts_of_few_rows_encoded(fmt, T, skew):
    E, N, K = 64, 288, 160
    plan, (_, _, _, source), a, bc, bs, _ = _rows_case(T, 1, E, N, K, False, 0.1, skew, seed=3, scale=-3)
    args = (a.codes, a.scales, bc, bs, plan, N, K)
    y32 = mx.gemm_experts(*args, act=mx.ACT_GELU, dtype=F32).y
    for want_y in (False, True):
        out = mx.gemm_experts(*args, act=mx.ACT_GELU, want_y=want_y, fmt=fmt)
        mx.check_status()
        assert_encoding_of(out.codes, out.scales, y32.cpu().numpy(), fmt == mx.FMT_MXFP8, "y")
        assert not out.codes[dev(source) < 0].any()


def test_many_experts_captured_and_replayed_with_another_plan():
    T, picks, E, N, K = 40, 2, 64, 264, 288
    weights = _experts_operand(E, N, K, False, 1)[:2]
    index, x = [dev(routing(T, picks, E, seed, 0.1, 1)) for seed in (1, 2)], torch.randn(T, K, device="cuda")

    def call(i):
        plan = mx.expert_plan(i, E)
        rows = mx.expert_dispatch(x, plan, fmt=mx.FMT_MXFP4)
        return mx.gemm_experts(rows.codes, rows.scales, *weights, plan, N, K, act=mx.ACT_RELU).y
    want = [call(i) for i in index]
    held = index[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(held)
    for i, w in ((1, want[1]), (0, want[0])):
        held.copy_(index[i])
        y.fill_(7)
        graph.replay()
        assert torch.equal(y, w)
    mx.check_status()
