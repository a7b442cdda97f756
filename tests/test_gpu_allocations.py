"""What the torch entry points allocate is seen by dispatch modes and the profiler, and
filled where torch fills fresh memory; the results are the same."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.product_testutil import Operand, dev, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


class Allocations(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func._schema.name == "aten::empty":
            self.made.append(out.data_ptr())
        return out


def _calls():
    """A call and the outputs that it allocates one by one (a plan's parts share one allocation)."""
    x, w = torch.randn(40, 256, device="cuda"), torch.ones(256, device="cuda")
    index, weights = dev(routing(40, 2, 3, 1)), torch.rand(40, 2, device="cuda")
    plan = mx.expert_plan(index, 3)
    a, b = Operand(40, 256, False, 1), Operand(64, 256, False, 2)
    return {
        "rmsnorm": lambda: mx.rmsnorm(x, w, x, fmt=mx.FMT_MXFP4),
        "swiglu": lambda: mx.swiglu(x, fmt=mx.FMT_MXFP8),
        "gemm_bias_act": lambda: mx.gemm_bias_act(a.codes, a.scales, b.codes, b.scales, 40, 64, 256, want_z=True, fmt=mx.FMT_MXFP4),
        "bias_act_backward": lambda: mx.bias_act_backward(x, x, mx.ACT_SILU),
        "expert_plan": lambda: mx.expert_plan(index, 3),
        "expert_dispatch": lambda: mx.expert_dispatch(x, plan, fmt=mx.FMT_MXFP4),
        "expert_combine_backward": lambda: mx.expert_combine_backward(x, torch.zeros(plan.source.numel(), 256, device="cuda"), plan, weights),
    }


NAMES = ["rmsnorm", "swiglu", "gemm_bias_act", "bias_act_backward", "expert_plan", "expert_dispatch", "expert_combine_backward"]


def _tensors(out):
    return [t for t in out if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_a_dispatch_mode_sees_the_outputs(name):
    call = _calls()[name]
    want = _tensors(call())
    with Allocations() as seen:
        got = _tensors(call())
    outputs = [got[0]] if name == "expert_plan" else got
    assert {t.data_ptr() for t in outputs} <= set(seen.made), (len(outputs), len(seen.made))
    assert all(torch.equal(u, v) for u, v in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_the_profiler_lists_them_and_a_deterministic_run_fills_them(name):
    call = _calls()[name]
    want = _tensors(call())
    torch.use_deterministic_algorithms(True)
    try:
        assert torch.utils.deterministic.fill_uninitialized_memory
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
            got = _tensors(call())
    finally:
        torch.use_deterministic_algorithms(False)
    names = [e.name for e in prof.events()]
    made = 1 if name == "expert_plan" else len(got)
    assert names.count("aten::empty") >= made and sum(n.startswith("aten::fill_") for n in names) >= made, names
    assert all(torch.equal(u, v) for u, v in zip(got, want))
