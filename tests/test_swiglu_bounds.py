"""The error bound that SwiGLU's kernel states for its sigmoid from the hardware's 2^x
and reciprocal, by the same sequence of fp32 roundings on the host, with 2^x two
units and the reciprocal one unit in the last place off either way (what their
documentation allows)."""
import numpy as np

from tests.block_testutil import U, sigmoid64

F = np.float32


def _off(v, units):
    for _ in range(abs(units)):
        v = np.nextafter(v, F(np.inf if units > 0 else 0), dtype=F)
    return v


def test_fast_sigmoid_stays_within_its_stated_bound():
    g = np.concatenate([np.linspace(-80, 80, 1_000_001), np.random.default_rng(1).uniform(-80, -8, 1_000_000),
                        [-44.42355]]).astype(F)
    z = g * F(float.fromhex("-0x1.715476p+0"))
    exact, units = sigmoid64(g.astype(np.float64)), 7 + 1.23 * np.abs(g.astype(np.float64))
    worst = np.zeros(g.shape)
    for a in (-2, 0, 2):
        d = F(1) + _off(np.exp2(z.astype(np.float64)).astype(F), a)
        for b in (-1, 0, 1):
            s = _off((1 / d.astype(np.float64)).astype(F), b)
            worst = np.maximum(worst, np.abs(s - exact) / (exact * U))
    assert (worst <= units).all()
    # log2(e)'s own rounding counts: the other terms alone do not bound it
    assert (worst > 7 + np.abs(g)).any()
