"""What the products with an epilogue and by expert refuse of torch tensors (shapes,
types, sizes of operands), before anything is launched: on a GPU machine, since the call's
device is current by then."""
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.test_product_host import BF16, E, F32, I32, K, N, NAMES, P, PICKS, PLAN, T, U8, _calls, _operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


def _on_gpu(shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


WORKSPACE = {"bias_act_backward": 2, "expert_plan": 1, "linear_experts_wgrad": 6}   # of any type
# Tensors whose last size is the call's to choose: columns of the first, the number of choices.
FREE = {"expert_plan": {0}, "expert_dispatch": {0, 3}, "expert_combine": {0}, "expert_combine_backward": {0}, "gemm_experts": {6},
        "gemm_experts_wgrad": {6}, "linear_experts_wgrad": {0, 1, 4}}


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_of_the_cpu_or_of_another_shape_or_type_is_refused(name):
    call, shapes = _calls()[name]
    for i, (shape, dtype) in enumerate(shapes):
        if WORKSPACE.get(name) == i:
            continue
        tensors = [_on_gpu(s, t) for s, t in shapes]
        others = [torch.empty(shape, dtype=dtype), _on_gpu(shape, torch.float64)]
        if i not in FREE.get(name, ()):
            others.append(_on_gpu(shape[:-1] + (max(1, shape[-1] - (8 if len(shape) > 1 else 1)),), dtype))
        for other in others:
            with pytest.raises(ValueError):
                call(tensors[:i] + [other] + tensors[i + 1:])


def test_other_dtypes_and_a_missing_z_are_refused():
    for call in (lambda: mx.gemm_bias_act(*[_on_gpu(s, t) for s, t in _operands(T, N)], T, N, K, dtype=torch.float16),
                 lambda: mx.gemm_bias_act(*[_on_gpu(s, t) for s, t in _operands(T, N)], T, N, K, operands=0),
                 lambda: mx.bias_act_backward(_on_gpu((T, N)), act=mx.ACT_GELU),
                 lambda: mx.expert_plan(_on_gpu((T, PICKS), I32), 0),
                 lambda: mx.quantize_experts(_on_gpu((E, N, K), F32)),
                 lambda: mx.expert_combine_backward(_on_gpu((T, K)), None, mx.ExpertPlan(*(_on_gpu(s, t) for s, t in PLAN)), _on_gpu((T, PICKS)))):
        with pytest.raises(ValueError):
            call()
