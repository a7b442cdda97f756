"""The operators between the GEMMs refuse a call whose tensors lie on several devices
before anything is launched, and a stream of another device.  The tensors have sizes
and devices and no memory, so no GPU is needed."""
from types import SimpleNamespace

import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build

F32, BF16 = torch.float32, torch.bfloat16


class Placed(torch.Tensor):
    """A tensor that is said to be on a device; its address is null."""

    @staticmethod
    def __new__(cls, shape, dtype, device):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on a tensor without memory")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _at(shape, dtype=F32, device="cuda:0"):
    return Placed(shape, dtype, device)


T, K = 4, 64
NORM = dict(x=(T, K), weight=(K,), residual=(T, K), out_h=(T, K))
NORM_BACKWARD = dict(dy=(T, K), h=(T, K), weight=(K,), rstd=(T,), dres=(T, K), ws=(4096,), out_dx=(T, K))
GLU_BACKWARD = dict(dy=(T, K), gu=(T, 2 * K), out=(T, 2 * K))
CALLS = [(mx.rmsnorm, NORM, name) for name in NORM] + [(mx.rmsnorm_backward, NORM_BACKWARD, name) for name in NORM_BACKWARD]
CALLS += [(mx.swiglu_backward, GLU_BACKWARD, name) for name in GLU_BACKWARD]


@pytest.mark.parametrize("call,shapes,name", CALLS, ids=lambda v: getattr(v, "__name__", v if isinstance(v, str) else ""))
def test_one_tensor_elsewhere_is_refused(call, shapes, name):
    args = {k: _at(s, BF16 if k == "out" else F32, "cuda:1" if k == name else "cuda:0") for k, s in shapes.items()}
    with pytest.raises(ValueError, match="must be on cuda:[01] like"):
        call(**args)


@pytest.mark.parametrize("where", range(3))
def test_gradients_on_two_devices_are_refused(where):
    grads = [_at((100,), device="cuda:1" if i == where else "cuda:0") for i in range(3)]
    same = [_at((100,)) for _ in range(3)]
    for call in (lambda: mx.grad_norm(grads), lambda: mx.clip_grads(grads, 1.0),
                 lambda: mx.clip_grads(same, 1.0, out=grads),
                 lambda: mx.clip_grads(same, 1.0, ws=_at((1 << 20,), torch.uint8, "cuda:1")),
                 lambda: mx.grad_norm(same, ws=_at((1 << 20,), torch.uint8, "cuda:1"))):
        with pytest.raises(ValueError, match="must be on cuda:[01] like"):
            call()


def test_a_stream_of_another_device_is_refused():
    stream = SimpleNamespace(device=torch.device("cuda:1"))
    x, w = _at((T, K)), _at((K,))
    for call in (lambda: mx.rmsnorm(x, w, stream=stream), lambda: mx.rmsnorm_backward(x, x, w, _at((T,)), stream=stream),
                 lambda: mx.swiglu(x, stream=stream), lambda: mx.swiglu_backward(x, _at((T, 2 * K)), stream=stream),
                 lambda: mx.grad_norm([x], stream=stream), lambda: mx.clip_grads(iter([x]), 1.0, stream=stream)):
        with pytest.raises(ValueError, match="stream must be on cuda:0"):
            call()
