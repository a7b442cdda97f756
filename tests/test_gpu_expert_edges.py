"""Calls by expert that the documentation allows and few programs make."""
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build

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
