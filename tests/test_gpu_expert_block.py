"""The example of a block of experts: it runs, gives the same bits twice, and its
gradients are those of the block in 64 bits up to the products' FP4.

Tolerance: an E2M1 value within a block is off by a quarter of itself at most and, over
the magnitudes of a Gaussian block, by about 0.1 of itself in the mean square; a
product of two such operands is off by sqrt(2) 0.1 = 0.15 relatively, and a gradient
here is at most four such products deep: sqrt(4) 0.15 = 0.3, held to 0.5."""
import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


def test_training_runs_and_repeats():
    from examples.expert_block_step import train
    args = dict(tokens=160, width=96, hidden=128, experts=5, picks=2, steps=4, report=lambda line: None)
    losses, norms = train(**args)
    assert np.isfinite(losses).all() and np.isfinite(norms).all()
    assert train(**args) == (losses, norms)


def test_gradients():
    from examples.expert_block_step import NAMES, ExpertBlock
    T, K, H, E, k = 256, 128, 192, 6, 2
    block = ExpertBlock(K, H, E, k, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    block.norm += 0.2 * torch.randn(K, generator=g, device="cuda")
    block.b1 += 0.2 * torch.randn(H, generator=g, device="cuda")
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    dout = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    out, kept = block.forward(x)
    dx, grads = block.backward(dout, kept)
    mx.check_status()
    index = kept[3]

    leaves = [w.double().requires_grad_() for w in block.weights()]
    norm, router, w1, b1, w2, gate_up, down = leaves
    X = x.double().requires_grad_()
    n = X * (X.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * norm
    y = X + torch.nn.functional.gelu(n @ w1.T + b1) @ w2.T
    weights = torch.softmax((n @ router.T).gather(1, index), 1)
    for j in range(k):
        e = index[:, j]
        gate, up = torch.einsum("tk,tfk->tf", n, gate_up[e]).chunk(2, -1)
        y = y + weights[:, j:j + 1] * torch.einsum("tf,tkf->tk", torch.nn.functional.silu(gate) * up, down[e])
    true = torch.autograd.grad(y, [X, *leaves], dout.double())
    for name, got, ref in zip(("out", "x") + NAMES, (out, dx, *grads), (y, *true)):
        off = ((got.double() - ref).norm() / ref.norm()).item()
        assert off < 0.5, (name, off)
