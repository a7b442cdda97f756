"""Calls by expert that the documentation allows and few programs make."""
import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.mx_testutil import GEMM_TOL
from tests.product_testutil import Operand, assert_within, device_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


def _filled(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------- no choices
@pytest.mark.parametrize("fmt", [0, mx.FMT_MXFP4, mx.FMT_MXFP8])
@pytest.mark.parametrize("T", [0, 1, 700])
def test_tokens_without_choices_are_not_read_and_leave_rows_of_zeros(T, fmt):
    L, P, K = mx.lib(), 256, 1056
    source = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    y, codes, scales = _filled(2 * P * K), _filled(P * K if fmt == mx.FMT_MXFP8 else P * K // 2), _filled(L.mx_scales_bytes(P, K))
    encoded = (codes.data_ptr(), scales.data_ptr()) if fmt else (None, None)
    assert L.mx_expert_dispatch(None, 1, K, None, source.data_ptr(), T, 0, P, K, y.data_ptr(), fmt, *encoded, None) == 0
    mx.check_status()
    assert not y.any() and (not fmt or not (codes.any() or scales.any()))
    y.fill_(0xA5)
    assert L.mx_expert_combine_backward(None, 1, K, None, 0, K, None, source.data_ptr(), None, T, 0, P, K, y.data_ptr(), fmt, *encoded, None, None) == 0
    mx.check_status()
    assert not y.any()
    res = torch.randn(max(T, 1), K, device="cuda")
    out = torch.empty_like(res)
    assert L.mx_expert_combine(None, 0, K, None, None, T, 0, P, K, res.data_ptr(), 1, K, out.data_ptr(), 1, None) == 0
    mx.check_status()
    assert T == 0 or torch.equal(out, res)


def test_tokens_without_choices_from_torch():
    T, K = 37, 96
    plan = mx.expert_plan(torch.empty(T, 0, dtype=torch.int32, device="cuda"), 3)
    assert plan.offsets.tolist() == [0] * 4 and plan.slot.shape == (T, 0) and plan.source.numel() == 0
    res = torch.randn(T, K, device="cuda")
    assert mx.expert_dispatch(res, plan).y.shape == (0, K)
    assert torch.equal(mx.expert_combine(torch.empty(0, K, device="cuda"), plan, residual=res), res)
    mx.check_status()


@pytest.mark.parametrize("T,picks", [(0, 2), (37, 0)])
def test_a_layer_s_gradients_of_no_rows(T, picks):
    E, K, F, bf16 = 3, 128, 64, torch.bfloat16
    plan = mx.expert_plan(torch.empty(T, picks, dtype=torch.int64, device="cuda"), E)
    dy, w = torch.ones(T, K, device="cuda"), torch.empty(T, picks, device="cuda")
    weights = torch.randn(E, K, F, device="cuda").to(bf16)
    g = mx.expert_combine_backward(dy, torch.empty(0, K, device="cuda"), plan, w, fmt=mx.FMT_MXFP4)
    assert g.y.shape == (0, K) and g.dweights.shape == (T, picks)
    dh = mx.gemm_experts(g.codes, g.scales, *mx.quantize_experts(weights, mx.CONTRACT_ROWS), plan, F, K)
    assert dh.y.shape == (0, F)
    dz = mx.bias_act_backward(dh.y, torch.empty(0, F, dtype=bf16, device="cuda"), mx.ACT_GELU, fmt=mx.FMT_MXFP4)
    assert dz.dz.shape == (0, F) and not dz.dbias.any()
    assert not mx.linear_experts_wgrad(g.y, dz.dz, plan, out=torch.ones(E, K, F, device="cuda")).any()
    assert torch.equal(mx.expert_combine(g.y, plan, residual=dy), dy)
    with pytest.raises(ValueError, match="weights"):
        mx.expert_combine_backward(dy, torch.empty(0, K, device="cuda"), plan, None)
    mx.check_status()


@pytest.mark.parametrize("experts", [513, 1 << 40, (1 << 63) - 1])
def test_too_many_experts_are_refused_before_memory_is_taken(experts):
    index = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    with pytest.raises(mx.MXError):
        mx.expert_plan(index, experts)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


# ---------------------------------------------------------------------------- plans of one's own
# Blocks of 32 columns, blocks of 128, tiles.
KERNELS = {"blocks": (12, 96), "lines": (12, 2080), "tiles": (3, 2080)}


def _placed(E, before, taken, behind):
    """A plan whose first segment begins `before` rows in, with `taken[e]` rows for expert e and `behind` rows after the last; its rows with a token."""
    offsets, real = [before], []
    for n in taken:
        real += range(offsets[-1], offsets[-1] + n)
        offsets.append(offsets[-1] + -(-n // 128) * 128)
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    source = torch.full((offsets[-1] + behind,), -1, dtype=torch.int32, device="cuda")
    source[real] = whole(range(len(real)))
    return mx.ExpertPlan(whole(offsets), whole(list(taken) + [0] * (E - len(taken))), whole(real)[:, None], source), real


def _product(plan, E, N, K, operands, **kw):
    """Products of ones by expert e + 1: (outputs in memory that held other values, the row's values)."""
    P = plan.source.numel()
    ones = lambda lines: (torch.full((lines, K if operands == mx.FMT_MXFP8 else K // 2), 0x38 if operands == mx.FMT_MXFP8 else 0x22, dtype=torch.uint8,  # noqa: E731
                                     device="cuda"))
    scales = lambda lines, byte: torch.full((mx.scales_bytes(lines, K),), byte, dtype=torch.uint8, device="cuda")  # noqa: E731
    b = torch.cat([scales(N, 127 + e % 4) for e in range(E)])
    L = mx.lib()
    y, z = torch.full((P, N), float("nan"), device="cuda"), torch.full((P, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    codes, s = _filled(P * N // (1 if operands == mx.FMT_MXFP8 else 2)), _filled(mx.scales_bytes(P, N))
    rows, weights = (ones(P), scales(P, 127)), (ones(E * N), b)
    assert L.mx_gemm_experts(*(t.data_ptr() for t in (*rows, *weights)), operands, plan.offsets.data_ptr(), plan.counts.data_ptr(), E, P, N, K, None, 0, 0,
                             y.data_ptr(), 1, z.data_ptr(), operands, codes.data_ptr(), s.data_ptr(), None) == 0
    mx.check_status()
    return y, z, codes.view(P, -1), s.view(P // 128, -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(P, -1)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("operands", [mx.FMT_MXFP4, mx.FMT_MXFP8])
@pytest.mark.parametrize("before,behind", [(128, 0), (256, 128), (0, 256)])
def test_rows_around_the_segments_are_zero(kernel, operands, before, behind):
    E, N = KERNELS[kernel]
    K, taken = 64, [5, 0, 130]
    plan, real = _placed(E, before, taken + [0] * (E - 3), behind)
    y, z, codes, scales = _product(plan, E, N, K, operands)
    want = torch.zeros_like(y)
    want[real[:5]] = K * 1.0
    want[real[5:]] = K * 4.0
    assert torch.equal(y, want) and torch.equal(z, want.bfloat16())
    other = torch.ones(y.shape[0], dtype=torch.bool, device="cuda")
    other[real] = False
    assert not codes[other].any() and not scales[other].any() and bool(codes[real].all())


BACKWARDS = {"to and fro": lambda E, P: [0, P] * E, "overlapping": lambda E, P: [0, 256, 128] + [P] * E, "at the end": lambda E, P: [128] * E + [0],
             "ends before the rows": lambda E, P: [0, P] + [-128] * E}


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("operands", [mx.FMT_MXFP4, mx.FMT_MXFP8])
@pytest.mark.parametrize("which", list(BACKWARDS))
def test_offsets_that_go_backwards_hold_no_rows(kernel, operands, which):
    E, N = KERNELS[kernel]
    P = 640
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = mx.ExpertPlan(whole(BACKWARDS[which](E, P)[:E + 1]), whole([100] * E), whole([[0]]), whole([-1] * P))
    for out in _product(plan, E, N, 64, operands):
        assert not out.any()


# ---------------------------------------------------------------------------- full capacity
def _all_in_one(E, n, N, K, fp8):
    """n rows of the last of E experts: operands, the plan, the rows alone and that expert's weights."""
    plan, (_, _, _, source) = device_plan(np.full((n, 1), E - 1, np.int32), E)
    rows, weights = Operand(source.size, K, fp8, 1, spread=9, lines_zero=source < 0), [Operand(N, K, fp8, 2 + e, spread=9) for e in range(E)]
    dense = Operand(n, K, fp8, 1)
    dense.codes, dense.scales = rows.codes[:n], rows.scales[:mx.scales_bytes(n, K)]
    return plan, rows, torch.cat([w.codes for w in weights]), torch.cat([w.scales for w in weights]), dense, weights[-1]


@pytest.mark.parametrize("E,n", [(1, 17), (1, 128), (2, 129), (4, 131)])
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
def test_few_experts_that_one_may_fill_have_the_dense_product_s_bits(E, n, fp8):
    # Rows of one expert enough for the dense product's tiles: the same kernel, so the same bits.
    N, K, operands = 264, 4128, mx.FMT_MXFP8 if fp8 else mx.FMT_MXFP4
    plan, rows, codes, scales, dense, b = _all_in_one(E, n, N, K, fp8)
    assert plan.source.numel() == 128 * E
    y = mx.gemm_experts(rows.codes, rows.scales, codes, scales, plan, N, K, dtype=torch.float32, operands=operands).y
    want = mx.gemm_bias_act(dense.codes, dense.scales, b.codes, b.scales, n, N, K, dtype=torch.float32, operands=operands).y
    mx.check_status()
    assert torch.equal(y[:n], want) and not y[n:].any()


@pytest.mark.parametrize("E,n", [(7, 7), (8, 8), (8, 135), (16, 143)])
@pytest.mark.parametrize("fp8", [False, True], ids=["mxfp4", "mxfp8"])
def test_a_full_capacity_of_one_expert_s_rows(E, n, fp8):
    N, K = 96, 288
    plan, rows, codes, scales, _, b = _all_in_one(E, n, N, K, fp8)
    assert plan.source.numel() == 128 * E
    y = mx.gemm_experts(rows.codes, rows.scales, codes, scales, plan, N, K, dtype=torch.float32, operands=mx.FMT_MXFP8 if fp8 else mx.FMT_MXFP4).y
    mx.check_status()
    a = rows.values[:n]
    assert_within(y[:n], a @ b.values.T, GEMM_TOL * (np.abs(a) @ np.abs(b.values).T), "y")
    assert not y[n:].any()
