"""What the products with an epilogue and the products by expert are measured on.

  linear         z = A B^T + bias, y = act(z) + residual, with A, B in MXFP4 or MXFP8; y in bf16 and / or as MXFP8 rows, z kept for the gradient
  act_bwd        its gradient: dz = dy * act'(z), dbias = sum over rows of dz
  dispatch       the order of the rows by expert (each expert's segment at a multiple of 128 rows), and the tokens' rows in that order, encoded
  experts        y = act(A B_e^T + bias_e) for the rows of each expert e; rows that belong to none are zero
  experts_wgrad  dW_e = dY^T X over the rows of each expert e
  combine        y = residual + sum over a token's choices of weight * row ("out"), and its gradient ("grad"): drow = weight * dy, dweight = dy . row

`run` computes them in plain torch where `own` is false, through the package where it is true.  Codes and scales come back as
the 8-bit floating types that they are, so as the values that they stand for; scales in the tiled order that the GEMM reads.
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPE = {"f32": F32, "bf16": BF16}
ACTS = ["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]
MOST = 8192 * 14336 * 4096  # products of the largest dense case


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # A few tokens of a decoding step through a projection with bias; an odd hidden size; joins the residual stream.
        {"name": "linear tokens", "op": "linear", "rows": 5, "cols": 4128, "depth": 2080, "operands": "mx8", "act": "silu", "bias": "bf16", "res": "bf16", "pad": 64, "z": False,
         "enc": False},
        # Training forward at the gate/up and down widths (T = 8192): y for the Wgrad, its encoding for the next product, z for the gradient.
        {"name": "linear train", "op": "linear", "rows": 8192, "cols": 14336, "depth": 4096, "operands": "mx4", "act": "gelu", "bias": "bf16", "res": None, "pad": 0, "z": True,
         "enc": True},
        # A small odd micro-batch's backward pass.
        {"name": "act_bwd small", "op": "act_bwd", "rows": 97, "cols": 2080, "dy": "bf16", "act": "relu2", "pad": 32},
        # Training backward at the same widths, from the Dgrad's fp32 result.
        {"name": "act_bwd train", "op": "act_bwd", "rows": 8192, "cols": 14336, "dy": "f32", "act": "gelu", "pad": 0},
        # A few tokens of a decoding step, sent to their experts.
        {"name": "dispatch tokens", "op": "dispatch", "rows": 9, "picks": 4, "experts": 16, "cols": 2080, "x": "bf16", "keep": False, "drop": 0.0, "skew": 1.0},
        # Training forward, many small experts: rows kept in bf16 for the Wgrad.
        {"name": "dispatch train", "op": "dispatch", "rows": 8192, "picks": 4, "experts": 64, "cols": 4096, "x": "bf16", "keep": True, "drop": 0.0, "skew": 0.5},
        # A few tokens of a decoding step, most experts without a row: the weights of the others are what is read.
        {"name": "experts tokens", "op": "experts", "rows": 12, "picks": 2, "experts": 64, "cols": 2048, "depth": 2048, "operands": "mx4", "act": "none", "bias": False, "drop": 0.0,
         "skew": 0.5},
        # Training forward of large experts, two for each token.
        {"name": "experts train", "op": "experts", "rows": 8192, "picks": 2, "experts": 8, "cols": 14336, "depth": 4096, "operands": "mx4", "act": "silu", "bias": True, "drop": 0.0,
         "skew": 0.3},
        # A small batch's weight gradients, several experts without a row, some choices dropped.
        {"name": "wgrad small", "op": "experts_wgrad", "rows": 301, "picks": 2, "experts": 16, "cols": 1408, "depth": 2080, "operands": "mx8", "drop": 0.1, "skew": 2.0},
        # Training backward of the large experts.
        {"name": "wgrad train", "op": "experts_wgrad", "rows": 8192, "picks": 2, "experts": 8, "cols": 14336, "depth": 4096, "operands": "mx4", "drop": 0.0, "skew": 0.3},
        # A small odd batch's rows back in the tokens' order, some choices dropped.
        {"name": "combine small", "op": "combine", "way": "out", "rows": 37, "picks": 8, "experts": 64, "cols": 1048, "row": "f32", "res": "bf16", "drop": 0.2, "skew": 1.0},
        # Training backward of that step: the rows' gradients and the router's.
        {"name": "combine grad", "op": "combine", "way": "grad", "rows": 8192, "picks": 4, "experts": 64, "cols": 4096, "row": "bf16", "res": "bf16", "drop": 0.0, "skew": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _size(rng, lo, hi):
    """A power of two half the time, else an odd number."""
    n = _log(rng, lo, hi)
    return 1 << (n.bit_length() - 1) if rng.random() < 0.5 else min(n | 1, max(1, hi))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "act_bwd", "dispatch", "experts", "experts", "experts_wgrad", "combine"])
    t = lambda: rng.choice(["f32", "bf16"])  # noqa: E731
    flag = lambda: rng.random() < 0.5  # noqa: E731
    act, pad, mx = rng.choice(ACTS), rng.choice([0, 0, 32, 64]), rng.choice(["mx4", "mx4", "mx8"])
    cols, depth = 32 * _size(rng, 2, 511), 32 * _size(rng, 2, 511)
    if op == "linear":
        rows = _size(rng, 1, min(16383, MOST // (cols * depth), (1 << 27) // cols))
        return {"op": op, "rows": rows, "cols": cols, "depth": depth, "operands": mx, "act": act, "bias": rng.choice([None, "f32", "bf16"]), "res": rng.choice([None, "f32", "bf16"]),
                "pad": pad, "z": flag(), "enc": flag()}
    if op == "act_bwd":
        return {"op": op, "rows": _size(rng, 1, min(16383, (1 << 26) // cols)), "cols": cols, "dy": t(), "act": act, "pad": pad}
    experts = _size(rng, 1, 128)
    picks = rng.randint(1, min(8, experts))
    c = {"op": op, "picks": picks, "experts": experts, "drop": rng.choice([0.0, 0.0, 0.1]), "skew": rng.choice([0.0, 0.5, 2.0]), "cols": cols}
    if op in ("dispatch", "combine"):
        c["rows"] = _size(rng, 1, min(16383, (1 << 26) // (cols * picks)))
        return {**c, "x": t(), "keep": flag()} if op == "dispatch" else {**c, "way": rng.choice(["out", "grad"]), "row": t(), "res": t()}
    while experts * cols * depth > 8 * 14336 * 4096:
        cols, depth = 32 * max(2, cols // 64), 32 * max(2, depth // 64)
    c.update(cols=cols, depth=depth, operands=mx, rows=_size(rng, 1, min(8191, MOST // (cols * depth * picks), (1 << 26) // (max(cols, depth) * picks))))
    return {**c, "act": act, "bias": flag()} if op == "experts" else c


def _capacity(c):
    """Rows that the experts' segments can take, each rounded up to 128."""
    n = c["rows"] * c["picks"]
    return (n + 127 * min(c["experts"], n)) // 128 * 128


def work(case):
    c, size = case, {"f32": 4, "bf16": 2, None: 0, "mx4": 0.5 + 1 / 32, "mx8": 1 + 1 / 32}
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "linear":
        m = size[c["operands"]]
        each = 2 + size[c["res"]] + (2 if c["z"] else 0) + (size["mx8"] if c["enc"] else 0)
        return {"bytes": (rows + cols) * c["depth"] * m + rows * cols * each + cols * size[c["bias"]], "flops": 2 * rows * cols * c["depth"]}
    if c["op"] == "act_bwd":
        return {"bytes": rows * cols * (size[c["dy"]] + 4) + 4 * cols, "flops": 20 * rows * cols}
    n = rows * c["picks"] * (1 - c["drop"])  # rows that an expert gets
    used = c["experts"] * (1 - (1 - 1 / c["experts"]) ** n)  # experts that get one
    if c["op"] == "dispatch":
        each = size["mx8"] + (2 if c["keep"] else 0)
        return {"bytes": rows * cols * size[c["x"]] + n * cols * each + 12 * n, "flops": 4 * rows * cols}
    if c["op"] == "experts":
        m = size[c["operands"]]
        return {"bytes": (n + used * cols) * c["depth"] * m + 2 * n * cols, "flops": 2 * n * cols * c["depth"]}
    if c["op"] == "experts_wgrad":
        return {"bytes": n * (cols + c["depth"]) * size[c["operands"]] + 4 * c["experts"] * cols * c["depth"], "flops": 2 * n * cols * c["depth"]}
    if c["way"] == "out":
        return {"bytes": cols * (n * size[c["row"]] + 2 * rows * size[c["res"]]), "flops": 2 * n * cols}
    return {"bytes": cols * (n * (size[c["row"]] + 2) + rows * size[c["res"]]), "flops": 3 * n * cols}


# ---------------------------------------------------------------------------------------------- inputs
def _made(g, rows, cols, pad=0, spread=1.0, outliers=False, tails=False):
    """Rows of cols, a slice of rows of cols + pad; activations have 1% of channels times 20, gradients heavy tails."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda") * spread
    if outliers:
        x *= torch.where(torch.rand(cols + pad, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    if tails:  # Student-t with 3 degrees of freedom, at the standard deviation `spread`
        chi = sum(torch.randn(rows, cols + pad, generator=g, device="cuda").square_() for _ in range(3))
        x = x / chi.clamp_(min=1e-4).sqrt_()
    return x[:, :cols]


def _tiled(byte):
    """Scale bytes [matrices, rows, blocks] in the GEMM's order: 512-byte atoms of 128 rows x 4 blocks, each matrix's rows and blocks padded with zeros."""
    p = torch.nn.functional.pad(byte, (0, -byte.shape[2] % 8, 0, -byte.shape[1] % 128))
    return p.view(p.shape[0], p.shape[1] // 128, 4, 32, p.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1)


def _block_scales(b, top_exponent):
    """E8M0 byte of each block [..., 32] and the power of two that takes the block to its codes' range."""
    top = b.abs().amax(-1)
    byte = torch.where(top > 0, torch.frexp(top).exponent + (127 - 1 - top_exponent), 0).clamp_(min=0)
    return byte.to(torch.uint8), torch.ldexp(torch.ones_like(top), 127 - byte)


def _mxfp8(y):
    """E4M3 codes and tiled E8M0 scales of fp32 rows [matrices, rows, columns], 32 columns to a scale."""
    b = y.unflatten(-1, (-1, 32))
    byte, inverse = _block_scales(b, 8)
    return (b * inverse[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(y.shape), _tiled(byte)


def _mxfp4(y):
    """The same with E2M1 codes, two to a byte: the first in the low half."""
    b = y.unflatten(-1, (-1, 32))
    byte, inverse = _block_scales(b, 2)
    v = b * inverse[..., None]
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    level = ((v / step).round_() * step).abs_().clamp_(max=6)
    code = torch.where(level < 2, 2 * level, torch.where(level < 4, 2 + level, 4 + 0.5 * level)).to(torch.uint8) | (v < 0).to(torch.uint8) << 3
    code = code.view(y.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, _tiled(byte)


def _operand(x, kind):
    """[matrices, rows, depth] as a product's operand (codes' bytes, scales' bytes)."""
    codes, scales = (_mxfp8 if kind == "mx8" else _mxfp4)(x)
    return codes.view(torch.uint8).flatten(0, 1), scales


def _routed(s, c, g):
    """Each token's experts, and the order of the rows that follows from them."""
    T, k, E = c["rows"], c["picks"], c["experts"]
    liked = torch.randn(E, generator=g, device="cuda") * c["skew"]
    score = liked + torch.distributions.utils.clamp_probs(torch.rand(T, E, generator=g, device="cuda")).log().neg().log().neg()
    top = score.topk(k, dim=1)
    s["experts"] = torch.where(torch.rand(T, k, generator=g, device="cuda") < c["drop"], -1, top.indices).to(torch.int32)
    s["weights"] = torch.softmax(top.values, 1)
    s.update(_ordered(s["experts"], c))
    s["longest"] = max(1, int(s["counts"].max()))


def _ordered(experts, c):
    """Rows by expert in the order of (token, choice), each expert's segment at a multiple of 128."""
    E, P = c["experts"], _capacity(c)
    e = experts.flatten().long()
    e = torch.where(e < 0, E, e)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device).index_add_(0, e, torch.ones_like(e))
    offsets = torch.nn.functional.pad(((counts[:E] + 127) // 128 * 128).cumsum(0), (1, 0))
    order = e.argsort(stable=True)
    by = e[order]
    first = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    at = torch.where(by < E, offsets[by] + torch.arange(e.numel(), device=e.device) - first[by], P)
    slot = torch.empty_like(e).index_copy_(0, order, torch.where(by < E, at, -1))
    source = torch.full((P + 1,), -1, dtype=torch.int64, device=e.device).index_copy_(0, at, order)
    return {"offsets": offsets.int(), "counts": counts[:E].int(), "slot": slot.view(experts.shape).int(), "source": source[:P].int()}


def prepare(case, seed):
    c, s = case, {"case": case}
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "linear":
        s["a"] = _operand(_made(g, rows, c["depth"], outliers=True)[None], c["operands"])
        s["b"] = _operand(_made(g, cols, c["depth"], spread=c["depth"] ** -0.5)[None], c["operands"])
        s["bias"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(TYPE[c["bias"]]) if c["bias"] else None
        s["res"] = _made(g, rows, cols + c["pad"]).to(TYPE[c["res"]])[:, :cols] if c["res"] else None
        return s
    if c["op"] == "act_bwd":
        s["dy"] = _made(g, rows, cols + c["pad"], spread=1e-3, tails=True).to(TYPE[c["dy"]])[:, :cols]
        s["z"] = _made(g, rows, cols, spread=1.5).to(BF16)
        return s
    _routed(s, c, g)
    P, E = _capacity(c), c["experts"]
    if c["op"] == "dispatch":
        s["x"] = _made(g, rows, cols, outliers=True).to(TYPE[c["x"]])
        return s
    real = (s["source"] >= 0)[:, None]
    if c["op"] == "experts":
        s["a"] = _operand(torch.where(real, _made(g, P, c["depth"], outliers=True), 0.0)[None], c["operands"])
        s["b"] = _operand((torch.randn(E, cols, c["depth"], generator=g, device="cuda") * c["depth"] ** -0.5), c["operands"])
        s["bias"] = 0.1 * torch.randn(E, cols, generator=g, device="cuda") if c["bias"] else None
    elif c["op"] == "experts_wgrad":
        s["a"] = _operand(torch.where(real, _made(g, P, cols, spread=1e-3, tails=True), 0.0).T.contiguous()[None], c["operands"])
        s["b"] = _operand(torch.where(real, _made(g, P, c["depth"], outliers=True), 0.0).T.contiguous()[None], c["operands"])
    else:
        s["rows"] = torch.where(real, _made(g, P, cols), 0.0).to(TYPE[c["row"]])
        s["res"] = _made(g, rows, cols, spread=2.0 if c["way"] == "out" else 1e-3).to(TYPE[c["res"]])  # the stream, or its gradient
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)(state, state["case"])


def _own(s, c):
    import mxfp4_precision_gb300 as mx
    act = {"none": mx.ACT_NONE, "relu": mx.ACT_RELU, "relu2": mx.ACT_RELU2, "gelu": mx.ACT_GELU, "gelu_tanh": mx.ACT_GELU_TANH, "silu": mx.ACT_SILU}
    fmt = {"mx4": mx.FMT_MXFP4, "mx8": mx.FMT_MXFP8}
    e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    if c["op"] == "linear":
        o = mx.gemm_bias_act(*s["a"], *s["b"], c["rows"], c["cols"], c["depth"], bias=s["bias"], act=act[c["act"]], residual=s["res"], want_z=c["z"],
                             fmt=mx.FMT_MXFP8 if c["enc"] else None, operands=fmt[c["operands"]])
        return {"y": o.y, "z": o.z, "codes": o.codes.view(e4m3) if c["enc"] else None, "scales": o.scales.view(e8m0) if c["enc"] else None}
    if c["op"] == "act_bwd":
        o = mx.bias_act_backward(s["dy"], s["z"], act=act[c["act"]])
        return {"dz": o.dz, "dbias": o.dbias}
    if c["op"] == "dispatch":
        plan = mx.expert_plan(s["experts"], c["experts"])
        o = mx.expert_dispatch(s["x"], plan, fmt=mx.FMT_MXFP8, want_y=c["keep"])
        return {"offsets": plan.offsets, "counts": plan.counts, "slot": plan.slot, "source": plan.source, "y": o.y, "codes": o.codes.view(e4m3), "scales": o.scales.view(e8m0)}
    plan = mx.ExpertPlan(s["offsets"], s["counts"], s["slot"], s["source"])
    if c["op"] == "experts":
        return {"y": mx.gemm_experts(*s["a"], *s["b"], plan, c["cols"], c["depth"], bias=s["bias"], act=act[c["act"]], operands=fmt[c["operands"]]).y}
    if c["op"] == "experts_wgrad":
        return {"dw": mx.gemm_experts_wgrad(*s["a"], *s["b"], plan, c["cols"], c["depth"], operands=fmt[c["operands"]])}
    if c["way"] == "out":
        return {"y": mx.expert_combine(s["rows"], plan, weights=s["weights"], residual=s["res"])}
    o = mx.expert_combine_backward(s["res"], s["rows"], plan, s["weights"])
    return {"drows": o.y, "dweights": o.dweights}


def _values(operand, matrices, rows, depth, kind):
    """A product's operand as fp32 [matrices, rows, depth]."""
    codes, scales = operand
    if kind == "mx8":
        v = codes.view(torch.float8_e4m3fn).to(F32)
    else:
        level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = level[torch.stack([codes & 15, codes >> 4], -1).int()]
    groups, atoms = -(-rows // 128), 2 * -(-depth // 256)
    byte = scales.view(matrices, groups, atoms, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(matrices, groups * 128, atoms * 4)[:, :rows, :depth // 32]
    return (v.view(matrices, rows, -1, 32) * torch.exp2(byte.to(F32) - 127)[..., None]).view(matrices, rows, depth)


def _activated(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "relu2":
        return z.clamp(min=0).square()
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2 * z.clamp(min=0)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        t = torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    return torch.ones_like(z)


def _by_expert(s, c):
    """Rows [experts, longest] of each segment, whether they are real, and where they go (past the end if not)."""
    n = torch.arange(s["longest"], device="cuda")
    real = n < s["counts"][:, None]
    at = s["offsets"][:-1, None].long() + n
    return torch.where(real, at, 0), real, torch.where(real, at, _capacity(c)).flatten()


def _plain(s, c):
    rows, cols, P = c["rows"], c["cols"], _capacity(c) if "experts" in c else 0
    if c["op"] == "linear":
        a, b = _values(s["a"], 1, rows, c["depth"], c["operands"])[0], _values(s["b"], 1, cols, c["depth"], c["operands"])[0]
        z = a @ b.T
        z = z if s["bias"] is None else z + s["bias"].float()
        y = _activated(z, c["act"])
        y = y if s["res"] is None else y + s["res"].float()
        codes, scales = _mxfp8(y[None]) if c["enc"] else (None, None)
        return {"y": y.to(BF16), "z": z.to(BF16) if c["z"] else None, "codes": codes[0] if c["enc"] else None,
                "scales": scales.view(torch.float8_e8m0fnu) if c["enc"] else None}
    if c["op"] == "act_bwd":
        dz = s["dy"].float() * _slope(s["z"].float(), c["act"])
        return {"dz": dz.to(BF16), "dbias": dz.sum(0)}
    if c["op"] == "dispatch":
        plan = _ordered(s["experts"], c)
        at = torch.where(plan["slot"] < 0, P, plan["slot"]).flatten().long()
        y = torch.zeros(P + 1, cols, device="cuda").index_copy_(0, at, s["x"].float().repeat_interleave(c["picks"], 0))[:P]
        codes, scales = _mxfp8(y[None])
        return {**plan, "y": y.to(BF16) if c["keep"] else None, "codes": codes[0], "scales": scales.view(torch.float8_e8m0fnu)}
    if c["op"] == "experts":
        at, real, to = _by_expert(s, c)
        z = torch.bmm(_values(s["a"], 1, P, c["depth"], c["operands"])[0][at], _values(s["b"], c["experts"], cols, c["depth"], c["operands"]).mT)
        z = z if s["bias"] is None else z + s["bias"][:, None]
        return {"y": torch.zeros(P + 1, cols, dtype=BF16, device="cuda").index_copy_(0, to, _activated(z, c["act"]).to(BF16).flatten(0, 1))[:P]}
    if c["op"] == "experts_wgrad":
        at, real, _ = _by_expert(s, c)
        a, b = _values(s["a"], 1, cols, P, c["operands"])[0], _values(s["b"], 1, c["depth"], P, c["operands"])[0]
        return {"dw": torch.bmm((a[:, at] * real).transpose(0, 1), b[:, at].permute(1, 2, 0))}
    there, at = s["slot"] >= 0, s["slot"].clamp(min=0).long()
    w = torch.where(there, s["weights"], 0.0)[:, :, None]
    picked = s["rows"].float()[at]
    if c["way"] == "out":
        return {"y": (s["res"].float() + (w * picked).sum(1)).to(s["res"].dtype)}
    dy = s["res"].float()[:, None]
    to = torch.where(there, at, P).flatten()
    drows = torch.zeros(P + 1, cols, device="cuda").index_copy_(0, to, (w * dy).flatten(0, 1))[:P]
    return {"drows": drows.to(BF16), "dweights": torch.where(there, (dy * picked).sum(2), 0.0)}


# ---------------------------------------------------------------------------------------------- in 64 bits
def _exact_operand(operand, matrices, rows, depth, kind):
    """The operand's values by the formats' definitions: sign, exponent and mantissa of each code, times its block's power of two."""
    codes, scales = operand[0].reshape(matrices, rows, -1).int(), operand[1].int()
    if kind == "mx8":
        sign, e, m, bias, width = codes >> 7, codes >> 3 & 15, codes & 7, 7, 8.0
    else:
        codes = torch.stack([codes & 15, codes >> 4], -1).reshape(matrices, rows, depth)
        sign, e, m, bias, width = codes >> 3, codes >> 1 & 3, codes & 1, 1, 2.0
    v = torch.where(e == 0, m.double() / width * 2.0 ** (1 - bias), (1 + m.double() / width) * torch.exp2((e - bias).double()))
    v = torch.where(sign == 1, -v, v)
    r, k = torch.arange(rows, device=codes.device)[:, None], torch.arange(depth // 32, device=codes.device)[None, :]
    atoms = 2 * -(-depth // 256)
    place = (r // 128 * atoms + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4
    each = -(-rows // 128) * atoms * 512
    byte = scales.view(matrices, each)[:, place.flatten()].view(matrices, rows, depth // 32)
    return v * torch.exp2((byte - 127).double()).repeat_interleave(32, 2)


def _exact_act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act in ("relu", "relu2"):
        up = torch.relu(z)
        return (up, (z > 0).double()) if act == "relu" else (up * up, 2 * up)
    if act == "gelu":
        below = torch.special.ndtr(z)
        return z * below, below + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        sig = torch.sigmoid(z)
        return z * sig, sig + z * sig * (1 - sig)
    u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)  # (1 + tanh(u / 2)) / 2 = sigmoid(u)
    sig = torch.sigmoid(u)
    return z * sig, sig + z * sig * (1 - sig) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)


def _exact8(y):
    """Codes' values and scales' values by the format's definition: the nearest of E4M3's values (ties to even), eight binades under the scale's top."""
    rows, cols = y.shape
    v = y.reshape(rows, cols // 32, 32)
    top = v.abs().max(-1).values
    binade = lambda t: torch.frexp(t).exponent.double() - 1  # noqa: E731  (exact at powers of two, where a logarithm may fall short)
    power = torch.where(top > 0, binade(top) - 8, -127.0).clamp(min=-127)
    v = v * torch.exp2(-power).unsqueeze(-1)
    step = torch.exp2(binade(v.abs().clamp(min=2.0 ** -6)) - 3)
    codes = (torch.round(v / step) * step).clamp(-448, 448).reshape(rows, cols)
    groups, atoms = -(-rows // 128), 2 * -(-cols // 256)
    full = torch.full((groups * 128, atoms * 4), 2.0 ** -127, dtype=torch.float64, device=y.device)
    full[:rows, :cols // 32] = torch.exp2(power)
    r, b = torch.meshgrid(torch.arange(groups * 128, device=y.device), torch.arange(atoms * 4, device=y.device), indexing="ij")
    flat = torch.empty(full.numel(), dtype=torch.float64, device=y.device)
    flat[(r // 128 * atoms + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = full
    return codes, flat


def exact(case, seed):
    s, c = prepare(case, seed), case
    rows, cols = c["rows"], c["cols"]
    if c["op"] == "linear":
        a, b = (_exact_operand(s[k], 1, n, c["depth"], c["operands"])[0] for k, n in (("a", rows), ("b", cols)))
        z = torch.einsum("rd,cd->rc", a, b)
        if s["bias"] is not None:
            z = z + s["bias"].double().unsqueeze(0)
        y, _ = _exact_act(z, c["act"])
        if s["res"] is not None:
            y = y + s["res"].double()
        codes, scales = _exact8(y) if c["enc"] else (None, None)
        return {"y": y, "z": z if c["z"] else None, "codes": codes, "scales": scales}
    if c["op"] == "act_bwd":
        dz = s["dy"].double() * _exact_act(s["z"].double(), c["act"])[1]
        return {"dz": dz, "dbias": torch.einsum("rc->c", dz)}
    # Each expert's entries, in the order of (token, choice), from the routing alone.
    P, flat = _capacity(c), s["experts"].flatten().tolist()
    mine = [[] for _ in range(c["experts"])]
    for i, e in enumerate(flat):
        if e >= 0:
            mine[e].append(i)
    start = [0]
    for m in mine:
        start.append(start[-1] + -(-len(m) // 128) * 128)
    slot = [-1] * len(flat)
    for e, m in enumerate(mine):
        for n, i in enumerate(m):
            slot[i] = start[e] + n
    if c["op"] == "dispatch":
        y = torch.zeros(P, cols, dtype=torch.float64, device="cuda")
        for e, m in enumerate(mine):
            if m:
                y[start[e]:start[e] + len(m)] = s["x"].double()[torch.tensor(m, device="cuda") // c["picks"]]
        codes, scales = _exact8(y)
        return {"offsets": None, "counts": None, "slot": None, "source": None, "y": y if c["keep"] else None, "codes": codes, "scales": scales}
    if c["op"] == "experts":
        a = _exact_operand(s["a"], 1, P, c["depth"], c["operands"])[0]
        y = torch.zeros(P, cols, dtype=torch.float64, device="cuda")
        for e, m in enumerate(mine):
            if m:
                each = -(-cols // 128) * 2 * -(-c["depth"] // 256) * 512
                b = _exact_operand((s["b"][0][e * cols:(e + 1) * cols], s["b"][1][e * each:(e + 1) * each]), 1, cols, c["depth"], c["operands"])[0]
                z = a[start[e]:start[e] + len(m)] @ b.T
                y[start[e]:start[e] + len(m)] = _exact_act(z if s["bias"] is None else z + s["bias"][e].double(), c["act"])[0]
        return {"y": y}
    if c["op"] == "experts_wgrad":
        a, b = _exact_operand(s["a"], 1, cols, P, c["operands"])[0], _exact_operand(s["b"], 1, c["depth"], P, c["operands"])[0]
        return {"dw": torch.stack([a[:, start[e]:start[e] + len(m)] @ b[:, start[e]:start[e] + len(m)].T for e, m in enumerate(mine)])}
    where = torch.tensor(slot, device="cuda").view(rows, c["picks"])
    w, out = torch.where(where >= 0, s["weights"].double(), 0.0), s["res"].double()
    if c["way"] == "out":
        for j in range(c["picks"]):
            out = out + w[:, j:j + 1] * s["rows"][where[:, j].clamp(min=0)].double()
        return {"y": out}
    drows, dw = torch.zeros(P, cols, dtype=torch.float64, device="cuda"), torch.zeros(rows, c["picks"], dtype=torch.float64, device="cuda")
    for j in range(c["picks"]):
        has = where[:, j] >= 0
        drows[where[has, j]] = w[has, j:j + 1] * out[has]
        dw[has, j] = torch.einsum("tc,tc->t", out[has], s["rows"][where[has, j]].double())
    return {"drows": drows, "dweights": dw}
