"""What the operators between the GEMMs of a training step are measured on.

A step of a quantised linear layer needs, beside its GEMMs:

  norm      h = x + r, y = h * rstd * w with rstd = 1 / sqrt(mean(h^2) + eps), and y's MXFP8 encoding
            (E4M3 codes, one E8M0 scale for 32 columns) that the next Fprop GEMM reads
  norm_bwd  its gradient: dx = rstd * (dy * w - h * rstd^2 * mean(dy * w * h)) + dres, dw = sum over rows of dy * h * rstd
  glu       y = silu(g) * u over the halves of a gate/up product, with the same encoding
  glu_bwd   its gradient: dg = dy * u * s * (1 + g * (1 - s)), du = dy * g * s, with s = sigmoid(g)
  clip      the L2 norm over all gradients and each of them times min(1, max_norm / (norm + 1e-6))

`run` computes them in plain torch where `own` is false, through the package where it is true.  Codes and scales come back as
the 8-bit floating types that they are, so as the values that they stand for; the scales in the tiled order that the GEMM reads.
"""
import math
import random

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPE = {"f32": F32, "bf16": BF16}
EPS = 1e-5


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One token of a decoding step: the attention's projection joins the residual stream, then the next GEMM's operand.
        {"name": "norm token", "op": "norm", "rows": 1, "cols": 4096, "x": "f32", "stream": "bf16", "keep": False, "pad": 0},
        # A ragged batch of tokens and a hidden size that fills neither a warp nor the scales' tiles.
        {"name": "norm ragged", "op": "norm", "rows": 777, "cols": 4128, "x": "bf16", "stream": "bf16", "keep": True, "pad": 64},
        # Training forward at the o_proj workload (T = 8192): y is kept in bf16 for the Wgrad.
        {"name": "norm train", "op": "norm", "rows": 8192, "cols": 4096, "x": "f32", "stream": "bf16", "keep": True, "pad": 0},
        # A whole prompt before the fused QKV product (T = 16384), nothing kept.
        {"name": "norm prompt", "op": "norm", "rows": 16384, "cols": 4096, "x": "f32", "stream": "bf16", "keep": False, "pad": 0},
        # A small odd micro-batch's backward pass.
        {"name": "norm_bwd small", "op": "norm_bwd", "rows": 97, "cols": 2080, "dy": "bf16", "stream": "bf16", "pad": 0},
        # Training backward at the same workload: the Dgrad's fp32 result and the residual stream's gradient.
        {"name": "norm_bwd train", "op": "norm_bwd", "rows": 8192, "cols": 4096, "dy": "f32", "stream": "bf16", "pad": 0},
        # A few sequences decoding: the down projection's operand.
        {"name": "glu tokens", "op": "glu", "rows": 4, "cols": 14336, "gu": "bf16", "keep": False, "pad": 0},
        # Training forward at the down_proj workload, from the GEMM's fp32 result, y kept for the Wgrad.
        {"name": "glu train", "op": "glu", "rows": 8192, "cols": 14336, "gu": "f32", "keep": True, "pad": 0},
        # A small odd micro-batch's backward pass.
        {"name": "glu_bwd small", "op": "glu_bwd", "rows": 333, "cols": 1760, "dy": "bf16", "gu": "bf16", "pad": 32},
        # Training backward at the down_proj workload.
        {"name": "glu_bwd train", "op": "glu_bwd", "rows": 8192, "cols": 14336, "dy": "f32", "gu": "f32", "pad": 0},
        # An adapter's or a set of norms' gradients: many small tensors of odd sizes, packed one after another.
        {"name": "clip small", "op": "clip", "set": "odd", "count": 64, "most": 20000, "shapes": 1, "grad": "bf16", "to": "bf16", "std": 0.02},
        # One layer's weight gradients (QKV, o_proj, gate/up, down_proj, two norms) as the Wgrads leave them, handed on in bf16.
        {"name": "clip layer", "op": "clip", "set": "layer", "count": 6, "most": 0, "shapes": 0, "grad": "f32", "to": "bf16", "std": 1e-3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A power of two half the time, else an odd number."""
    n = _log(rng, lo, hi)
    return 1 << (n.bit_length() - 1) if rng.random() < 0.5 else n | 1


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "glu", "glu_bwd", "clip"])
    t = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    flag = lambda: rng.random() < 0.5  # noqa: E731
    pad = rng.choice([0, 0, 32, 64])
    if op == "clip":
        return {"op": op, "set": "odd", "count": _log(rng, 1, 300), "most": _log(rng, 1000, 600000), "shapes": rng.randrange(1 << 30), "grad": t(), "to": t(),
                "std": rng.choice([1e-6, 1e-3, 0.02])}
    cols = 32 * _size(rng, 2, 511)
    rows = _size(rng, 1, min(16383, (1 << 25) // cols))
    if op == "norm":
        return {"op": op, "rows": rows, "cols": cols, "x": t(), "stream": t(), "keep": flag(), "pad": pad}
    if op == "norm_bwd":
        return {"op": op, "rows": rows, "cols": cols, "dy": t(), "stream": t(), "pad": pad}
    if op == "glu":
        return {"op": op, "rows": rows, "cols": cols, "gu": t(), "keep": flag(), "pad": pad}
    return {"op": op, "rows": rows, "cols": cols, "dy": t(), "gu": t(), "pad": pad}


def _sizes(c):
    if c["set"] == "layer":
        return [6144 * 4096, 4096 * 4096, 28672 * 4096, 4096 * 14336, 4096, 4096]
    r = random.Random(c["shapes"])
    return [_log(r, 1, c["most"]) for _ in range(c["count"])]


def work(case):
    c, size = case, {"f32": 4, "bf16": 2}
    if c["op"] == "clip":
        n = sum(_sizes(c))
        return {"bytes": n * (size[c["grad"]] + size[c["to"]]) + 4, "flops": 3 * n}
    n, rows, cols = c["rows"] * c["cols"], c["rows"], c["cols"]
    if c["op"] == "norm":  # x, the stream in and out, codes, scales, y, w, rstd
        return {"bytes": n * (size[c["x"]] + 2 * size[c["stream"]] + 1 + 1 / 32 + (2 if c["keep"] else 0)) + 2 * cols + 4 * rows, "flops": 8 * n}
    if c["op"] == "norm_bwd":  # dy, h, the stream's gradient in and out, w, rstd, dw
        return {"bytes": n * (size[c["dy"]] + 3 * size[c["stream"]]) + 6 * cols + 4 * rows, "flops": 10 * n}
    if c["op"] == "glu":
        return {"bytes": n * (2 * size[c["gu"]] + 1 + 1 / 32 + (2 if c["keep"] else 0)), "flops": 10 * n}
    return {"bytes": n * (size[c["dy"]] + 2 * size[c["gu"]] + 4), "flops": 16 * n}


# ---------------------------------------------------------------------------------------------- inputs
def _made(g, rows, cols, kind, pad=0, spread=1.0, outliers=False, tails=False):
    """A rows x cols matrix of the type, a slice of rows of cols + pad; activations have 1% of channels times 20, gradients heavy tails."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda") * spread
    if outliers:
        x *= torch.where(torch.rand(cols + pad, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    if tails:  # Student-t with 3 degrees of freedom, at the standard deviation `spread`
        chi = sum(torch.randn(rows, cols + pad, generator=g, device="cuda").square_() for _ in range(3))
        x = x / chi.clamp_(min=1e-4).sqrt_()
    return x.to(TYPE[kind])[:, :cols]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "clip":
        sizes = _sizes(c)
        s["grads"] = [(torch.randn(n, generator=g, device="cuda") * c["std"]).to(TYPE[c["grad"]]) for n in sizes]
        s["flat"] = torch.zeros(sum(sizes), dtype=TYPE[c["to"]], device="cuda")
        s["outs"] = list(s["flat"].split(sizes))  # a bucket's slices, at whatever element they begin
        return s
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "norm":
        s["x"] = _made(g, rows, cols, c["x"], c["pad"], 1.0, outliers=True)
        s["r"] = _made(g, rows, cols, c["stream"], 0, 2.0, outliers=True)
    if c["op"] == "norm_bwd":
        s["dy"] = _made(g, rows, cols, c["dy"], c["pad"], 1e-3, tails=True)
        s["h"] = _made(g, rows, cols, c["stream"], 0, 2.0, outliers=True)
        s["dres"] = _made(g, rows, cols, c["stream"], 0, 1e-3, tails=True)
        s["rstd"] = (s["h"].double().square().mean(-1) + EPS).rsqrt().float()
    if c["op"] in ("norm", "norm_bwd"):
        s["w"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(BF16)
        return s
    if c["op"] == "glu_bwd":
        s["dy"] = _made(g, rows, cols, c["dy"], 0, 1e-3, tails=True)
    s["gu"] = _made(g, rows, 2 * cols, c["gu"], c["pad"])
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)(state, state["case"])


def _own(s, c):
    import mxfp4_precision_gb300 as mx
    if c["op"] == "norm":
        o = mx.rmsnorm(s["x"], s["w"], residual=s["r"], eps=EPS, fmt=mx.FMT_MXFP8, want_y=c["keep"])
        return {"h": o.h, "y": o.y, "codes": o.codes.view(torch.float8_e4m3fn), "scales": o.scales.view(torch.float8_e8m0fnu), "rstd": o.rstd}
    if c["op"] == "norm_bwd":
        dx, dw = mx.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dres=s["dres"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "glu":
        o = mx.swiglu(s["gu"], fmt=mx.FMT_MXFP8, want_y=c["keep"])
        return {"y": o.y, "codes": o.codes.view(torch.float8_e4m3fn), "scales": o.scales.view(torch.float8_e8m0fnu)}
    if c["op"] == "glu_bwd":
        return {"dgu": mx.swiglu_backward(s["dy"], s["gu"])}
    return {"norm": mx.clip_grads(s["grads"], 1.0, out=s["outs"]), "clipped": s["flat"]}


def _tiled(byte, rows):
    """Scale bytes [rows, blocks] in the GEMM's order: 512-byte atoms of 128 rows x 4 blocks, rows and blocks padded with zeros."""
    blocks = byte.shape[1]
    p = torch.nn.functional.pad(byte, (0, -blocks % 8, 0, -rows % 128))
    return p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _mxfp8(y):
    """E4M3 codes and E8M0 scales of fp32 rows, 32 columns to a scale: the exponent of the block's largest magnitude, less 8."""
    b = y.view(y.shape[0], -1, 32)
    top = b.abs().amax(-1)
    byte = torch.where(top > 0, torch.frexp(top).exponent + (127 - 8 - 1), 0).clamp_(min=0)
    inverse = ((254 - byte) << 23).to(torch.int32).view(F32)
    codes = (b * inverse[:, :, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(y.shape)
    return codes, _tiled(byte.to(torch.uint8), y.shape[0]).view(torch.float8_e8m0fnu)


def _plain(s, c):
    if c["op"] == "norm":
        h = s["x"].float() + s["r"].float()
        rstd = (h.square().mean(-1) + EPS).rsqrt()
        y = h * rstd[:, None] * s["w"].float()
        codes, scales = _mxfp8(y)
        return {"h": h.to(s["r"].dtype), "y": y.to(BF16) if c["keep"] else None, "codes": codes, "scales": scales, "rstd": rstd}
    if c["op"] == "norm_bwd":
        dy, h, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
        xhat = h * r
        a = dy * s["w"].float()
        dx = r * (a - xhat * (a * xhat).mean(-1, keepdim=True)) + s["dres"].float()
        return {"dx": dx.to(s["h"].dtype), "dw": (dy * xhat).sum(0)}
    if c["op"] == "glu":
        g, u = s["gu"].float().chunk(2, -1)
        y = g / (1 + torch.exp(-g)) * u
        codes, scales = _mxfp8(y)
        return {"y": y.to(BF16) if c["keep"] else None, "codes": codes, "scales": scales}
    if c["op"] == "glu_bwd":
        g, u = s["gu"].float().chunk(2, -1)
        dy, sg = s["dy"].float(), 1 / (1 + torch.exp(-g))
        return {"dgu": torch.cat([dy * u * sg * (1 + g * (1 - sg)), dy * g * sg], -1).to(BF16)}
    flat = torch.cat(s["grads"]).float()
    norm = flat.square().sum().sqrt()
    s["flat"].copy_(flat * (1.0 / (norm + 1e-6)).clamp(max=1))
    return {"norm": norm.view(1), "clipped": s["flat"]}


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    d = lambda k: s[k].double()  # noqa: E731
    if c["op"] == "clip":
        flat = torch.cat([x.double() for x in s["grads"]])
        norm = torch.linalg.vector_norm(flat)
        return {"norm": norm.reshape(1), "clipped": flat * torch.clamp(1.0 / (norm + 1e-6), max=1.0)}
    if c["op"] == "norm":
        h = d("x") + d("r")
        mean = torch.einsum("rc,rc->r", h, h) / c["cols"]
        y = h / torch.sqrt(mean + EPS).unsqueeze(1) * d("w")
        codes, scales = _exact8(y)
        return {"h": h, "y": y if c["keep"] else None, "codes": codes, "scales": scales, "rstd": 1 / torch.sqrt(mean + EPS)}
    if c["op"] == "norm_bwd":
        r, h = d("rstd").unsqueeze(1), d("h")
        gw = d("dy") * d("w")
        along = torch.einsum("rc,rc->r", gw, h).unsqueeze(1) / c["cols"]
        return {"dx": gw * r - h * along * r ** 3 + d("dres"), "dw": torch.einsum("rc,rc->c", d("dy"), h * r)}
    gate, up = d("gu")[:, :c["cols"]], d("gu")[:, c["cols"]:]
    sig = torch.sigmoid(gate)
    if c["op"] == "glu":
        y = gate * sig * up
        codes, scales = _exact8(y)
        return {"y": y if c["keep"] else None, "codes": codes, "scales": scales}
    dy = d("dy")
    return {"dgu": torch.cat([dy * up * (sig + gate * sig * (1 - sig)), dy * gate * sig], 1)}


def _exact8(y):
    """Codes' values and scales' values by the format's definition: the nearest of E4M3's values (ties to even), eight binades under the scale's top."""
    rows, cols = y.shape
    v = y.reshape(rows, cols // 32, 32)
    top = v.abs().max(-1).values
    power = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 8, -127.0).clamp(min=-127)
    v = v * torch.exp2(-power).unsqueeze(-1)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    codes = (torch.round(v / step) * step).clamp(-448, 448).reshape(rows, cols)
    groups, atoms = -(-rows // 128), 2 * -(-cols // 256)
    full = torch.full((groups * 128, atoms * 4), 2.0 ** -127, dtype=torch.float64, device=y.device)
    full[:rows, :cols // 32] = torch.exp2(power)
    r, b = torch.meshgrid(torch.arange(groups * 128, device=y.device), torch.arange(atoms * 4, device=y.device), indexing="ij")
    flat = torch.empty(full.numel(), dtype=torch.float64, device=y.device)
    flat[(r // 128 * atoms + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = full
    return codes, flat
