"""A layer of experts, forward and backward, on operands that the formats hold without
rounding: weights that pick a column each with a sign, values of E2M1, weights of the choices
that are one power of two an expert.  A block of 32 such values is encoded exactly whatever its
largest, every sum is of multiples of 1/8 below 2^17, and y and dx are multiples of 1/4 below
64, which bf16 holds; so all outputs equal the 64-bit ones."""
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.product_testutil import dev, routing

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


def _values(g, *shape):
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return level[torch.randint(0, 8, shape, generator=g)] * (1 - 2 * torch.randint(0, 2, shape, generator=g))


def _pickers(g, E, rows, cols):
    """[E, rows, cols], one +-1 in each row and at most one in each column up to min(rows, cols)."""
    w = torch.zeros(E, rows, cols)
    for e in range(E):
        n = min(rows, cols)
        r, c = torch.randperm(rows, generator=g)[:n], torch.randperm(cols, generator=g)[:n]
        w[e, r, c] = 1.0 - 2 * torch.randint(0, 2, (n,), generator=g)
    return w


def _encoded(w, operands, down):
    """[E, rows, columns] as gemm_experts' B: lines are the rows, or (down) the columns."""
    if operands == mx.FMT_MXFP4:
        return mx.quantize_experts(w, mx.CONTRACT_ROWS if down else mx.CONTRACT_COLS)
    return mx.quantize_experts(w if down else w.mT.contiguous(), mx.CONTRACT_ROWS, operands=operands)


@pytest.mark.parametrize("operands", [mx.FMT_MXFP4, mx.FMT_MXFP8], ids=["mxfp4", "mxfp8"])
# Tiles; blocks of 128 columns; blocks of 32 columns.
@pytest.mark.parametrize("T,picks,E,K,F,drop", [(300, 2, 5, 160, 288, 0.1), (700, 3, 4, 288, 96, 0.0), (40, 1, 64, 288, 544, 0.1), (5, 2, 16, 96, 160, 0.0)])
def test_a_layer_and_its_gradients(T, picks, E, K, F, drop, operands):
    g = torch.Generator().manual_seed(T)
    x, d_out = (_values(g, T, K).cuda().to(BF16) for _ in range(2))
    w1, w2 = _pickers(g, E, F, K).cuda().to(BF16), _pickers(g, E, K, F).cuda().to(BF16)
    index = dev(routing(T, picks, E, T, drop))
    power = torch.tensor([1.0, 2.0, 0.5], device="cuda")
    w = torch.where(index >= 0, power[(index.long() % 3)], 5.0)

    plan = mx.expert_plan(index, E)
    rows = mx.expert_dispatch(x, plan, fmt=operands)
    h = mx.gemm_experts(rows.codes, rows.scales, *_encoded(w1, operands, False), plan, F, K, act=mx.ACT_RELU, want_z=True, fmt=operands, operands=operands)
    out = mx.gemm_experts(h.codes, h.scales, *_encoded(w2, operands, False), plan, K, F, operands=operands)
    y = mx.expert_combine(out.y, plan, w, x)
    back = mx.expert_combine_backward(d_out, out.y, plan, w, fmt=operands)
    dh = mx.gemm_experts(back.codes, back.scales, *_encoded(w2, operands, True), plan, F, K, operands=operands)
    dw2 = mx.linear_experts_wgrad(back.y, h.y, plan, operands=operands, rot=mx.ROT_NONE)
    dz = mx.bias_act_backward(dh.y, h.z, mx.ACT_RELU, fmt=operands)
    drows = mx.gemm_experts(dz.codes, dz.scales, *_encoded(w1, operands, True), plan, K, F, operands=operands)
    dw1 = mx.linear_experts_wgrad(dz.dz, rows.y, plan, operands=operands, rot=mx.ROT_NONE)
    dx = mx.expert_combine(drows.y, plan, residual=d_out)
    mx.check_status()

    leaves = [t.double().requires_grad_() for t in (x, w1, w2, w)]
    X, W1, W2, R = leaves
    want = X
    for j in range(picks):
        e, there = index[:, j].long().clamp(min=0), (index[:, j] >= 0)[:, None]
        hidden = torch.relu(torch.einsum("tk,tfk->tf", X, W1[e]))
        want = want + torch.where(there, R[:, j:j + 1] * torch.einsum("tf,tkf->tk", hidden, W2[e]), 0.0)
    true = torch.autograd.grad(want, leaves, d_out.double())
    for got, ref, name in ((y, want, "y"), (dx, true[0], "dx"), (dw1, true[1], "dw1"), (dw2, true[2], "dw2"), (back.dweights, true[3], "dweights")):
        assert ref.abs().max() > 0 and torch.equal(got.double(), ref), (name, (got.double() - ref).abs().max().item())
