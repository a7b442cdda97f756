"""Training steps of a block of experts with a shared dense part, every product in
MXFP4 and everything between them in this library's kernels but the router's small
product and softmax:

    n       = rmsnorm(x)                                    encoded for the products
    h       = gelu(n W1^T + b1),   s = x + h W2^T           the shared part
    plan    = each token's rows among its experts'          (expert_plan)
    rows    = n in the experts' order                       (expert_dispatch)
    a       = swiglu(rows Wgu_e^T),  o = a Wd_e^T           (gemm_experts)
    out     = s + sum over choices of weight * o            (expert_combine)

and back: expert_combine_backward, gemm_experts with the transposed weights,
linear_experts_wgrad, swiglu_backward, bias_act_backward, expert_combine (the dispatch's
gradient), rmsnorm_backward, clip_grads.

The loss is the squared distance of out from a fixed target; the weights take plain SGD
steps.  Run it on a GB300:

    python examples/expert_block_step.py [--tokens 512 --width 256 --hidden 256 --experts 8 --picks 2 --steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_precision_gb300 as mx  # noqa: E402

FP4 = mx.FMT_MXFP4
NAMES = ("norm", "router", "w1", "b1", "w2", "gate_up", "down")


class ExpertBlock:
    """Weights: fp32 masters; bf16 copies are encoded for the products of a step."""

    def __init__(self, width: int, hidden: int, experts: int, picks: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5  # noqa: E731
        self.norm = torch.ones(width, device="cuda")
        self.router = normal(experts, width)
        self.w1, self.b1, self.w2 = normal(hidden, width), torch.zeros(hidden, device="cuda"), normal(width, hidden)
        self.gate_up, self.down = normal(experts, 2 * hidden, width), normal(experts, width, hidden)
        self.width, self.hidden, self.experts, self.picks = width, hidden, experts, picks

    def weights(self):
        return [getattr(self, name) for name in NAMES]

    def forward(self, x, index=None):
        """(out bf16, what the backward pass needs) for x [T, width] in bf16; index: the experts of each token's choices,
        where they are given and not the router's first ones."""
        T, K, H = x.shape[0], self.width, self.hidden
        w1, w2, w_gu, w_d = (w.bfloat16() for w in (self.w1, self.w2, self.gate_up, self.down))
        n = mx.rmsnorm(x, self.norm, fmt=FP4)
        h = mx.gemm_bias_act(n.codes, n.scales, *mx.quantize(w1, mx.CONTRACT_COLS), T, H, K, bias=self.b1, act=mx.ACT_GELU, want_z=True,
                             fmt=FP4)
        s = mx.gemm_bias_act(h.codes, h.scales, *mx.quantize(w2, mx.CONTRACT_COLS), T, K, H, residual=x)
        logits = n.y.float() @ self.router.T
        if index is None:
            index = logits.topk(self.picks, 1).indices
        weights = torch.softmax(logits.gather(1, index), 1)
        plan = mx.expert_plan(index, self.experts)
        rows = mx.expert_dispatch(n.y, plan, fmt=FP4)
        gu = mx.gemm_experts(rows.codes, rows.scales, *mx.quantize_experts(w_gu), plan, 2 * H, K).y
        a = mx.swiglu(gu, fmt=FP4)
        o = mx.gemm_experts(a.codes, a.scales, *mx.quantize_experts(w_d), plan, K, H).y
        out = mx.expert_combine(o, plan, weights, s.y)
        return out, (x, n, h, index, weights, plan, rows, gu, a, o, w1, w2, w_gu, w_d)

    def backward(self, dout, kept):
        """(the gradient of x, the weights' in the order of NAMES) for out's gradient in bf16."""
        x, n, h, index, weights, plan, rows, gu, a, o, w1, w2, w_gu, w_d = kept
        K, H = self.width, self.hidden
        # The experts.
        g = mx.expert_combine_backward(dout, o, plan, weights, fmt=FP4)
        da = mx.gemm_experts(g.codes, g.scales, *mx.quantize_experts(w_d, mx.CONTRACT_ROWS), plan, H, K).y
        d_down = mx.linear_experts_wgrad(g.y, a.y, plan)
        dgu = mx.swiglu_backward(da, gu)
        d_rows = mx.gemm_experts(*mx.quantize(dgu, mx.CONTRACT_COLS), *mx.quantize_experts(w_gu, mx.CONTRACT_ROWS), plan, K, 2 * H).y
        d_gate_up = mx.linear_experts_wgrad(dgu, rows.y, plan)
        # The router.
        dw = g.dweights
        d_logits = torch.zeros(x.shape[0], self.experts, device=x.device)
        d_logits.scatter_(1, index, weights * (dw - (weights * dw).sum(1, keepdim=True)))
        # The shared part; its Dgrad joins the rows' and the router's gradients of n.
        dh = mx.linear_dgrad(dout, w2)
        d_w2 = mx.linear_wgrad(dout, h.y)
        b = mx.bias_act_backward(dh, h.z, mx.ACT_GELU)
        d_w1 = mx.linear_wgrad(b.dz, n.y)
        dn = mx.expert_combine(d_rows, plan, residual=mx.linear_dgrad(b.dz, w1))
        dn.addmm_(d_logits, self.router)
        dx, d_norm = mx.rmsnorm_backward(dn, x, self.norm, n.rstd, dres=dout)
        return dx, [d_norm, d_logits.T @ n.y.float(), d_w1, b.dbias, d_w2, d_gate_up, d_down]


def train(tokens: int = 512, width: int = 256, hidden: int = 256, experts: int = 8, picks: int = 2, steps: int = 20, lr: float = 0.2,
          max_norm: float = 1.0, seed: int = 0, report=print):
    """Losses and gradient norms of `steps` steps, as floats."""
    block = ExpertBlock(width, hidden, experts, picks, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    target = torch.tanh(x.float().roll(1, 1)) * 2
    losses, norms = [], []
    for _ in range(steps):
        out, kept = block.forward(x)
        diff = out.float() - target
        losses.append(diff.square().sum(-1).mean())
        _, grads = block.backward((diff * (2 / tokens)).bfloat16(), kept)
        norms.append(mx.clip_grads(grads, max_norm))
        for w, d in zip(block.weights(), grads):
            w.sub_(d, alpha=lr)
    mx.check_status()
    losses, norms = torch.stack(losses).tolist(), torch.cat(norms).tolist()
    for step, (loss, norm) in enumerate(zip(losses, norms)):
        report(f"step {step:3d}  loss {loss:9.4f}  gradient norm {norm:8.4f}")
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("width", 256), ("hidden", 256), ("experts", 8), ("picks", 2), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    train(**vars(ap.parse_args()))
