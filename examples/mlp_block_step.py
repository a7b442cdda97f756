"""Training steps of one transformer MLP block with every product in MXFP4 and
every operator between the products in this library's kernels:

    h, n   = rmsnorm(x, residual)           n encoded as the gate/up operand
    gu     = n Wgu^T                        fp32
    a      = swiglu(gu)                     encoded as the down operand
    out    = a Wd^T                         joins the stream: stream' = h + out
    da     = dout Wd,  dWd = dout^T a
    dgu    = swiglu_backward(da, gu)
    dn     = dgu Wgu,  dWgu = dgu^T n
    dx, dw = rmsnorm_backward(dn, h, dres)  dres: the stream's own gradient
    clip_grads([dWgu, dWd, dw])

The loss is the squared distance of stream' from a fixed target; the weights
take plain SGD steps.  Run it on a GB300:

    python examples/mlp_block_step.py [--tokens 512 --width 256 --hidden 704 --steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_precision_gb300 as mx  # noqa: E402


class MLPBlock:
    """Weights of a block: fp32 masters, bf16 copies for the products."""

    def __init__(self, width: int, hidden: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.norm = torch.ones(width, device="cuda")
        self.gate_up = normal(2 * hidden, width) * width ** -0.5
        self.down = normal(width, hidden) * hidden ** -0.5
        self.width, self.hidden = width, hidden

    def weights(self):
        return [self.gate_up, self.down, self.norm]

    def forward(self, x, stream):
        """(out fp32, what the backward pass needs); the stream is updated in place."""
        T = x.shape[0]
        n = mx.rmsnorm(x, self.norm, residual=stream, fmt=mx.FMT_MXFP4, out_h=stream)
        w_gu, w_d = self.gate_up.bfloat16(), self.down.bfloat16()
        gu = mx.gemm(n.codes, n.scales, *mx.quantize(w_gu, mx.CONTRACT_COLS), T, 2 * self.hidden,
                     self.width)
        a = mx.swiglu(gu, fmt=mx.FMT_MXFP4)
        out = mx.gemm(a.codes, a.scales, *mx.quantize(w_d, mx.CONTRACT_COLS), T, self.width, self.hidden)
        return out, (n, gu, a, w_gu, w_d)

    def backward(self, dout, dres, kept):
        """dout: the output's gradient in bf16; dres: the stream's.  Returns the stream's gradient before
        the block and [dgate_up, ddown, dnorm]."""
        n, gu, a, w_gu, w_d = kept
        da = mx.linear_dgrad(dout, w_d)
        d_down = mx.linear_wgrad(dout, a.y)
        dgu = mx.swiglu_backward(da, gu)
        dn = mx.linear_dgrad(dgu, w_gu)
        d_gate_up = mx.linear_wgrad(dgu, n.y)
        dx, d_norm = mx.rmsnorm_backward(dn, n.h, self.norm, n.rstd, dres=dres)
        return dx, [d_gate_up, d_down, d_norm]


def train(tokens: int = 512, width: int = 256, hidden: int = 704, steps: int = 20, lr: float = 0.5,
          max_norm: float = 1.0, seed: int = 0, report=print):
    """Losses and gradient norms of `steps` steps, as floats."""
    block = MLPBlock(width, hidden, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(tokens, width, generator=g, device="cuda")
    stream0 = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    target = torch.tanh((x + stream0.float()).roll(1, 1)) * 2
    losses, norms = [], []
    for step in range(steps):
        stream = stream0.clone()
        out, kept = block.forward(x, stream)
        diff = stream.float() + out - target
        losses.append(diff.square().sum(-1).mean())
        dout = (diff * (2 / tokens)).bfloat16()
        _, grads = block.backward(dout, dout, kept)
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
    for name, default in (("tokens", 512), ("width", 256), ("hidden", 704), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    train(**vars(ap.parse_args()))
