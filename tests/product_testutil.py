"""64-bit forms of the products with an epilogue and by expert, random operands,
and the tolerances their kernels are held to (shared by the GPU tests).

Tolerances: u = 2^-24.  An accumulator is within GEMM_TOL * sum |a| |b| of the
product (what every GEMM of this library is held to); bias and residual add a
rounding each.  An activation is within (16 + 4 x^2) u of its value relatively, from
mx_act.cuh: 2 ulp of 2^x and 1 of the reciprocal (8 u with the sum's rounding), four
further roundings, and the exponent's rounding, at most 3 |x|^2 u (gelu, its polynomial
within 3.7e-8 < u) or 3 u times 2.3 |x| + 0.1 |x|^3 <= 4 x^2 + 12 for gelu_tanh where its
tail is not below fp32's range (|x| < 10).  An error of z passes the activation with
its slope, at most 1.13 but for relu2 (2 |z|).  bf16 adds half a step, 2^-8 relatively.
"""
import math

import numpy as np
import torch
from scipy.special import erfc

import mxfp4_precision_gb300 as mx
import oracle
from tests.mx_testutil import GEMM_TOL, tile_scales

U, UB = 2.0 ** -24, 2.0 ** -8
ACTS = {"none": mx.ACT_NONE, "relu": mx.ACT_RELU, "relu2": mx.ACT_RELU2, "gelu": mx.ACT_GELU, "gelu_tanh": mx.ACT_GELU_TANH,
        "silu": mx.ACT_SILU}
E2M1 = np.array([oracle.e2m1_value(c) for c in range(16)])
E4M3 = np.array([oracle.e4m3_value(c) for c in range(256)])


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


class Operand:
    """Random codes and scales of [lines, k]: `values` in 64 bits, `codes` and `scales` (tiled) on the GPU."""

    def __init__(self, lines, k, fp8, seed, spread=3, scale=0, lines_zero=None):
        rng = np.random.default_rng(seed)
        if fp8:
            codes = rng.integers(0, 256, (lines, k), dtype=np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x38  # no NaN
            codes[(codes & 0x7F) > 0x5F] -= 0x20  # magnitudes up to 30, so that one code does not outweigh a row
        else:
            codes = rng.integers(0, 16, (lines, k), dtype=np.uint8)
        byte = rng.integers(127 - spread + scale, 128 + spread + scale, (lines, k // 32)).astype(np.uint8)
        if lines_zero is not None:
            codes[lines_zero] = 0
            byte[lines_zero] = 0
        self.byte, self.code = byte, codes
        self.values = (E4M3 if fp8 else E2M1)[codes] * np.repeat(np.exp2(byte.astype(np.float64) - 127), 32, 1)
        self.packed = codes if fp8 else codes[:, 0::2] | codes[:, 1::2] << 4
        self.codes, self.scales = dev(self.packed), dev(tile_scales(byte, lines, k)) if k else torch.empty(1, dtype=torch.uint8, device="cuda")
        if k == 0:
            self.codes = torch.empty((lines, 0), dtype=torch.uint8, device="cuda")


def sigmoid64(t):
    e = np.exp(-np.abs(t))
    return np.where(t >= 0, 1, e) / (1 + e)


def ndtr64(x):
    return 0.5 * erfc(-x / math.sqrt(2))


CT = 2 * math.sqrt(2 / math.pi)


def act64(name, x):
    if name == "relu":
        return np.maximum(x, 0)
    if name == "relu2":
        return np.maximum(x, 0) ** 2
    if name == "gelu":
        return x * ndtr64(x)
    if name == "gelu_tanh":
        return x * sigmoid64(CT * (x + 0.044715 * x ** 3))
    return x * sigmoid64(x) if name == "silu" else x


def slope64(name, x):
    if name == "relu":
        return (x > 0) * 1.0
    if name == "relu2":
        return 2 * np.maximum(x, 0)
    if name == "gelu":
        return ndtr64(x) + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        s = sigmoid64(CT * (x + 0.044715 * x ** 3))
        return s + x * s * (1 - s) * CT * (1 + 3 * 0.044715 * x * x)
    if name == "silu":
        s = sigmoid64(x)
        return s + x * s * (1 - s)
    return np.ones_like(x)


def act_bound(name, x):
    """Error of the activation itself at x (64-bit): relative, and fp32's subnormals."""
    return 0 if name == "none" else (16 + 4 * np.minimum(x * x, 200)) * U * np.abs(act64(name, x)) + 2.0 ** -140


def epilogue64(a, b, bias, act, res):
    """(z, its error bound, y, its error bound), before the outputs' own roundings."""
    acc, size = a @ b.T, np.abs(a) @ np.abs(b).T
    z = acc if bias is None else acc + bias
    ez = GEMM_TOL * size + U * np.abs(z)
    y = act64(act, z)
    lipschitz = {"none": 1, "relu": 1, "relu2": 2 * np.abs(z) + ez}.get(act, 1.13)
    ey = lipschitz * ez + act_bound(act, z)
    if res is not None:
        y = y + res
        ey = ey + U * np.abs(y)
    return z, ez, y, ey


def assert_within(got, ref, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; at {i}: got {got[i]!r}, want {ref[i]!r} "
                             f"within {np.broadcast_to(bound, ref.shape)[i]!r}")


def assert_output(got, ref, err, what):
    """An output rounded once from a value within err of ref."""
    half = UB if got.dtype == torch.bfloat16 else 0.0  # fp32's own rounding is in err
    assert_within(got, ref, err + half * (np.abs(ref) + err) + (2.0 ** -133 if half else 0), what)


def encode_of(y32, fp8):
    """(codes as stored, scale bytes [T, N / 32]) of fp32 rows, by the oracle's rules."""
    T, N = y32.shape
    blocks = y32.reshape(T, N // 32, 32)
    amax = np.abs(blocks).max(-1)
    byte = (oracle.scale_bytes_e4m3 if fp8 else oracle.scale_bytes)(amax.astype(np.float32))
    v = (blocks * np.exp2(127.0 - byte.astype(np.float64))[..., None]).astype(np.float32)
    c = (oracle.e4m3_rne if fp8 else oracle.e2m1_rne)(v).reshape(T, N)
    return (c if fp8 else c[:, 0::2] | c[:, 1::2] << 4), byte


def assert_encoding_of(codes, scales, y32, fp8, what):
    """codes and scales are, bit for bit, the encoding of the fp32 rows y32; the scales' padding is zero."""
    T, N = y32.shape
    want, byte = encode_of(y32, fp8)
    assert np.array_equal(scales.cpu().numpy(), tile_scales(byte, T, N)), f"{what}: scales"
    got = codes.cpu().numpy()
    # a code of -0 and one of 0 stand for the same value
    value = E4M3 if fp8 else None
    if fp8:
        assert np.array_equal(value[got], value[want]), f"{what}: codes"
    else:
        assert np.array_equal(E2M1[got & 15], E2M1[want & 15]) and np.array_equal(E2M1[got >> 4], E2M1[want >> 4]), f"{what}: codes"


def routing(T, picks, E, seed, drop=0.0, skew=0.5):
    """[T, picks] experts, distinct for a token, some dropped (-1)."""
    rng = np.random.default_rng(seed)
    score = rng.gumbel(size=(T, E)) + skew * rng.standard_normal(E)
    x = np.argsort(-score, 1)[:, :picks].astype(np.int32)
    x[rng.random((T, picks)) < drop] = -1
    return x


def plan64(index, E):
    """The plan as numpy arrays from its definition."""
    T, picks = index.shape
    n = T * picks
    P = (n + 127 * min(E, n)) // 128 * 128
    flat = index.reshape(-1)
    offsets, counts = np.zeros(E + 1, np.int32), np.zeros(E, np.int32)
    slot, source = np.full(n, -1, np.int32), np.full(P, -1, np.int32)
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        counts[e] = len(mine)
        slot[mine] = offsets[e] + np.arange(len(mine))
        source[offsets[e]:offsets[e] + len(mine)] = mine
        offsets[e + 1] = offsets[e] + -(-len(mine) // 128) * 128
    return offsets, counts, slot.reshape(T, picks), source


def device_plan(index, E):
    parts = plan64(index, E)
    return mx.ExpertPlan(*(dev(p) for p in parts)), parts
