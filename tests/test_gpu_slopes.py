"""The activations' slopes one by one: NaN, infinities and zeros, and the tails against
64-bit values, relative to the sizes of the slope's own terms.

Tolerances (u = 2^-24; h = the small part of act at -|x|).  2^y is within 2 ulp = 4 u, its
square 9 u.  The exponent t is within 4 u t for gelu_tanh (of its roundings, constants'
included, four add up), 3 u t for gelu and 2 u t for silu, which is as much relatively in
e = exp(-t): within d = 9 u + 4 u t.
  gelu       p(x) e and |x| phi each within d + 6 u (roundings, the polynomial's 3.7e-8)
  logistic   r = 1 / (1 + e) within d / 2 + 3 u, h = e r within 1.5 d + 4 u,
             |x| h r (1 + 3 c x^2) within 2 d + 12 u
and the sum rounds once more, twice where it is taken from 1.  So a slope is within (30 u + 8 u t)
of the sum of its terms' sizes, and u of itself.  Terms below fp32's normal range add 2^-138.
"""
import math

import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.product_testutil import ACTS, CT, U, dev, f64, ndtr64, sigmoid64, slope64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    mx.lib()


def _slope(act, x):
    """The kernel's slopes at x in fp32: one row's dz is its bias' gradient."""
    z = dev(np.asarray(x, np.float32)[None])
    out = mx.bias_act_backward(torch.ones_like(z), z, ACTS[act])
    mx.check_status()
    assert torch.equal(out.dz[0].nan_to_num(7), out.dbias.bfloat16().nan_to_num(7))
    return f64(out.dbias)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_slopes_of_nan_infinities_and_zeros(act, rows, dtype):
    x = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 3e38, -3e38, 1.0], device="cuda", dtype=dtype).expand(rows, 8).contiguous()
    out = mx.bias_act_backward(torch.full_like(x, 3.0), x, ACTS[act])
    mx.check_status()
    half, top = (3 * slope64(act, np.array([v]))[0] for v in (0.0, 1.0))
    finite = {"none": [3] * 8, "relu2": [math.nan, math.inf, 0, 0, 0, math.inf, 0, 6]}.get(act, [math.nan, 3, 0, half, half, 3, 0, top])
    for got in (out.dz[rows - 1], out.dbias / rows):
        # 2^-8 for bf16; relu2's 3 * 2 * 3e38 is beyond fp32
        np.testing.assert_allclose(f64(got), finite, rtol=2.0 ** -8, atol=0)


@pytest.mark.parametrize("act", [n for n in ACTS if n != "none"])
def test_slopes_over_their_range(act):
    x = np.concatenate([np.linspace(-14, 14, 8192), -np.geomspace(1e-30, 60, 1024), np.geomspace(1e-30, 60, 1024), -np.linspace(0.7, 0.8, 512)]).astype(np.float32)
    got, x = _slope(act, x), x.astype(np.float64)
    n = np.abs(x)
    if act == "gelu":
        t, terms = n * n / 2, ndtr64(-n) + n * np.exp(-n * n / 2) / math.sqrt(2 * math.pi)
    elif act in ("silu", "gelu_tanh"):
        t = n if act == "silu" else CT * (n + 0.044715 * n ** 3)
        h = sigmoid64(-t)
        terms = h + n * h * (1 - h) * (1 if act == "silu" else CT * (1 + 3 * 0.044715 * n * n))
    else:
        t = terms = 0 * n
    ref = slope64(act, x)
    bound = (30 + 8 * np.minimum(t, 200)) * U * terms + U * np.abs(ref) + 2.0 ** -138
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (act, int(bad.sum()), x[bad][:4], got[bad][:4], ref[bad][:4], bound[bad][:4])
