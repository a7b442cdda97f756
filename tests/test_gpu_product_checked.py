"""The bounds-checked build runs ragged shapes of the products with an epilogue
and by expert into buffers of exactly their size: no store may fall outside, and the
results equal the normal build's byte for byte."""
import ctypes

import numpy as np
import pytest
import torch

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build
from tests.product_testutil import Operand, dev, device_plan, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    build.build()
    normal, checked = mx.lib(), ctypes.CDLL(build.build(checked=True))
    for name in mx._binding.EXPORTED:
        fn = getattr(checked, name)
        fn.argtypes, fn.restype = getattr(normal, name).argtypes, getattr(normal, name).restype
    return normal, checked


def _buf(n):
    return torch.full((max(1, n),), 0xA5, dtype=torch.uint8, device="cuda")


def _same(libs, call):
    outs = []
    for L in libs:
        got = call(L)
        assert L.mx_check_status(None) == 0
        outs.append([t.cpu().numpy() for t in got])
    for u, v in zip(*outs):
        assert np.array_equal(u, v)


def _p(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (130, 288, 96), (515, 1056, 544)])
@pytest.mark.parametrize("fp8", [False, True])
def test_dense(libs, M, N, K, fp8):
    a, b = Operand(M, K, fp8, 1), Operand(N, K, fp8, 2)
    bias, res = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda").bfloat16()

    def call(L):
        y, z, c, s = _buf(4 * M * N), _buf(2 * M * N), _buf(M * N // 2), _buf(L.mx_scales_bytes(M, N))
        assert L.mx_gemm_bias_act(_p(a.codes), _p(a.scales), _p(b.codes), _p(b.scales), 2 if fp8 else 1, M, N, K, _p(bias), 1, 4, _p(res), 0, N, _p(y), 1,
                                  _p(z), 1, _p(c), _p(s), None) == 0
        return y, z, c, s
    _same(libs, call)


@pytest.mark.parametrize("T,N", [(1, 32), (97, 288), (1000, 1056)])
def test_gradient(libs, T, N):
    dy, z = torch.randn(T, N, device="cuda"), torch.randn(T, N, device="cuda").bfloat16()

    def call(L):
        dz, c, s, db, ws = _buf(2 * T * N), _buf(T * N), _buf(L.mx_scales_bytes(T, N)), _buf(4 * N), _buf(L.mx_bias_act_backward_workspace_bytes(T, N))
        assert L.mx_bias_act_backward(_p(dy), 1, N, _p(z), 0, N, 3, T, N, _p(dz), 2, _p(c), _p(s), _p(db), _p(ws), ws.numel(), None) == 0
        return dz, c, s, db
    _same(libs, call)


@pytest.mark.parametrize("T,picks,E,N,K", [(1, 1, 1, 32, 32), (130, 2, 5, 288, 160), (700, 3, 4, 1056, 96), (20, 2, 64, 288, 160)])
@pytest.mark.parametrize("fp8", [False, True])
def test_experts(libs, T, picks, E, N, K, fp8):
    plan, parts = device_plan(routing(T, picks, E, 1, 0.1), E)
    P, fmt = parts[3].size, 2 if fp8 else 1
    rows, weights = Operand(P, K, fp8, 1, lines_zero=parts[3] < 0), Operand(E * N, K, fp8, 2)
    if N % 128:
        each = [Operand(N, K, fp8, 3 + e) for e in range(E)]
        weights.codes, weights.scales = torch.cat([w.codes for w in each]), torch.cat([w.scales for w in each])
    down = [Operand(n, P, fp8, 4) for n in (N, K)]
    x, w, bias = torch.randn(T, K, device="cuda"), torch.rand(T, picks, device="cuda"), torch.randn(E, N, device="cuda")
    off, cnt, slot, src = (t.data_ptr() for t in plan)

    def call(L):
        y, z, c, s = _buf(4 * P * N), _buf(2 * P * N), _buf(P * N // 2 * fmt), _buf(L.mx_scales_bytes(P, N))
        assert L.mx_gemm_experts(_p(rows.codes), _p(rows.scales), _p(weights.codes), _p(weights.scales), fmt, off, cnt, E, P, N, K, _p(bias), 1, 5, _p(y), 1,
                                 _p(z), fmt, _p(c), _p(s), None) == 0
        dw = _buf(4 * E * N * K)
        assert L.mx_gemm_experts_wgrad(_p(down[0].codes), _p(down[0].scales), _p(down[1].codes), _p(down[1].scales), fmt, off, E, P, N, K, _p(dw), 1, None) == 0
        r, rc, rs = _buf(2 * P * K), _buf(P * K // 2), _buf(L.mx_scales_bytes(P, K))
        assert L.mx_expert_dispatch(_p(x), 1, K, slot, src, T, picks, P, K, _p(r), 1, _p(rc), _p(rs), None) == 0
        out = _buf(4 * T * K)
        assert L.mx_expert_combine(_p(r), 0, K, slot, _p(w), T, picks, P, K, _p(x), 1, K, _p(out), 1, None) == 0
        g, gc, gs, gw = _buf(2 * P * K), _buf(P * K), _buf(L.mx_scales_bytes(P, K)), _buf(4 * T * picks)
        assert L.mx_expert_combine_backward(_p(x), 1, K, _p(r), 0, K, slot, src, _p(w), T, picks, P, K, _p(g), 2, _p(gc), _p(gs), _p(gw), None) == 0
        return y, z, c, s, dw, r, rc, rs, out, g, gc, gs, gw
    _same(libs, call)


@pytest.mark.parametrize("T,picks,E", [(1, 1, 1), (300, 3, 64), (5000, 2, 512)])
def test_plan(libs, T, picks, E):
    index = dev(routing(T, picks, E, 2, 0.2))

    def call(L):
        P = L.mx_expert_rows(T, picks, E)
        parts = [_buf(4 * n) for n in (E + 1, E, T * picks, P)]
        ws = _buf(L.mx_expert_plan_workspace_bytes(T, picks, E))
        assert L.mx_expert_plan(_p(index), 4, T, picks, E, *(_p(t) for t in parts), _p(ws), ws.numel(), None) == 0
        return parts
    _same(libs, call)


def _guarded(n, kept):
    """n bytes between two lines of 4096 that must not change."""
    t = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    kept.append((t, n))
    return t.data_ptr() + 4096


OFFSETS = {
    "to and fro": lambda E, P, rng: np.array([0, P] * E)[:E + 1],
    "any": lambda E, P, rng: rng.integers(-2 ** 31, 2 ** 31, E + 1),
    "beyond the rows": lambda E, P, rng: np.sort(rng.integers(-P, 3 * P, E + 1)),
    "one too large": lambda E, P, rng: np.where(np.arange(E + 1) == E // 2, 2 ** 31 - 1, 128 * np.arange(E + 1)),
    "not whole groups": lambda E, P, rng: np.sort(rng.integers(0, P + 1, E + 1)),
}


@pytest.mark.parametrize("which", list(OFFSETS))
@pytest.mark.parametrize("E,P", [(512, 131072), (512, 65536), (512, 16384), (512, 4096), (3, 1024)])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_plan_of_any_content_stays_inside_the_buffers(libs, which, E, P, fp8):
    # No value of the outputs is asked for: what a plan like these means is not defined.
    rng = np.random.default_rng(E + P)
    T, picks, N, K, fmt = 200, 3, 160, 32, 2 if fp8 else 1
    whole = lambda n: dev(rng.integers(-2 ** 31, 2 ** 31, n).astype(np.int32))  # noqa: E731
    offsets = dev(OFFSETS[which](E, P, rng).astype(np.int32))
    counts, slot, source = whole(E), whole(T * picks), whole(P)
    slot[::2] %= P
    codes = lambda lines, k: torch.zeros(lines * k // (1 if fp8 else 2), dtype=torch.uint8, device="cuda")  # noqa: E731
    scales = lambda lines, k: torch.full((mx.lib().mx_scales_bytes(lines, k),), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    a, sa, b, sb = codes(P, K), scales(P, K), codes(E * N, K), scales(N, K).repeat(E)
    ta, tsa, tb, tsb = codes(K, P), scales(K, P), codes(N, P), scales(N, P)
    x, w, bias = torch.randn(T, K, device="cuda"), torch.rand(T, picks, device="cuda"), torch.randn(E, N, device="cuda")
    r = torch.randn(P, K, device="cuda").bfloat16()
    for L in libs:
        kept = []
        out = lambda n: _guarded(n, kept)  # noqa: E731
        rows = lambda n: out(P * n // (1 if fp8 else 2)), lambda n: out(L.mx_scales_bytes(P, n))  # noqa: E731
        assert L.mx_gemm_experts(_p(a), _p(sa), _p(b), _p(sb), fmt, _p(offsets), _p(counts), E, P, N, K, _p(bias), 1, 5, out(4 * P * N), 1, out(2 * P * N),
                                 fmt, rows[0](N), rows[1](N), None) == 0
        assert L.mx_gemm_experts_wgrad(_p(ta), _p(tsa), _p(tb), _p(tsb), fmt, _p(offsets), E, P, K, N, out(4 * E * K * N), 1, None) == 0
        assert L.mx_expert_dispatch(_p(x), 1, K, _p(slot), _p(source), T, picks, P, K, out(2 * P * K), fmt, rows[0](K), rows[1](K), None) == 0
        assert L.mx_expert_combine(_p(r), 0, K, _p(slot), _p(w), T, picks, P, K, _p(x), 1, K, out(4 * T * K), 1, None) == 0
        assert L.mx_expert_combine_backward(_p(x), 1, K, _p(r), 0, K, _p(slot), _p(source), _p(w), T, picks, P, K, out(2 * P * K), fmt, rows[0](K), rows[1](K),
                                            out(4 * T * picks), None) == 0
        assert L.mx_check_status(None) == 0
        for t, n in kept:
            assert bool((t[:4096] == 0xA5).all()) and bool((t[4096 + n:] == 0xA5).all())
