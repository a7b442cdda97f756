"""64-bit forms of the operators between the GEMMs and the tolerances their
fp32 kernels are held to (shared by the GPU tests).

Tolerances, from the kernels' arithmetic: u = 2^-24 is fp32's unit roundoff
and 2^-8 bf16's (8 significant bits).  A row's fp32 sum of K products, taken in parts of at most 64
terms a thread and then over threads as a tree, is off by at most
(64 + 16) u times the sum of magnitudes; half of that reaches rstd, and a
handful of further roundings follow: DELTA = 2^-17 (128 u) bounds an output's
relative error before its last rounding.
"""
import numpy as np
import torch

import oracle

U, UB = 2.0 ** -24, 2.0 ** -8
DELTA = 2.0 ** -17
TINY = 2.0 ** -126   # below fp32's (and bf16's) normal range errors are absolute


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def norm64(x, r, w, eps):
    """(h, y, rstd) in 64 bits from float64 arrays (r may be None)."""
    h = x if r is None else x + r
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h, h * rstd[:, None] * w, rstd


def norm_backward64(dy, h, w, rstd, dres):
    a, xh = dy * w, h * rstd[:, None]
    along = (a * xh).mean(-1, keepdims=True)
    return rstd[:, None] * (a - xh * along) + (0 if dres is None else dres), (dy * xh).sum(0)


def sigmoid64(g):
    return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def swiglu64(gu):
    g, u = np.split(gu, 2, -1)
    return g * sigmoid64(g) * u


def swiglu_backward64(dy, gu):
    g, u = np.split(gu, 2, -1)
    s = sigmoid64(g)
    return np.concatenate([dy * u * s * (1 + g * (1 - s)), dy * g * s], -1)


def assert_near(got, ref, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; at {i}: got "
                             f"{got[i]!r}, want {ref[i]!r} within {np.broadcast_to(bound, ref.shape)[i]!r}")


def canonical_scales(flat: np.ndarray, T: int, K: int):
    """Tiled scale bytes -> ([T, K/32], whether every padding byte is zero)."""
    groups, atoms = -(-T // 128), 2 * -(-K // 256)
    assert flat.size == groups * atoms * 512
    full = flat.reshape(groups, atoms, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(groups * 128, atoms * 4)
    pad = full.copy()
    pad[:T, :K // 32] = 0
    return full[:T, :K // 32], not pad.any()


def assert_encoded(codes, scales, y64, fmt, fp8: bool, what):
    """The encoding of y64 (finite): every scale byte and code lies between those of the value DELTA
    below and DELTA above; padding zero."""
    T, K = y64.shape
    bytes_, clean = canonical_scales(scales.cpu().numpy(), T, K)
    assert clean, f"{what}: scale padding not zero"
    blocks = y64.reshape(T, K // 32, 32)
    amax = np.abs(blocks).max(-1)
    scale_of = oracle.scale_bytes_e4m3 if fp8 else oracle.scale_bytes
    code_of = oracle.e4m3_rne if fp8 else oracle.e2m1_rne
    value = np.array([oracle.e4m3_value(c) if fp8 else oracle.e2m1_value(c) for c in range(256 if fp8 else 16)])
    lo, hi = (scale_of((amax * (1 + s * DELTA)).astype(np.float32)) for s in (-1, 1))
    assert ((bytes_ >= lo) & (bytes_ <= hi)).all(), f"{what}: scale bytes"
    v = blocks * np.exp2(127.0 - bytes_.astype(np.float64))[..., None]
    c = codes.cpu().numpy()
    if not fp8:
        c = np.stack([c & 15, c >> 4], -1)
    got = value[c.reshape(T, K // 32, 32)]
    ends = [value[code_of((v * (1 + s * DELTA)).astype(np.float32))] for s in (-1, 1)]
    lo, hi = np.minimum(*ends), np.maximum(*ends)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes, first at {np.argwhere(bad)[0]}"
