"""Row counts of plans at the ends of their range (host only)."""
import pytest

import mxfp4_precision_gb300 as mx
from mxfp4_precision_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


BIG = (1 << 31) - 1


@pytest.mark.parametrize("T,picks,experts,rows", [
    (BIG, BIG, 1 << 62, 0), (BIG, BIG, 1, 0), (BIG, 2, 8, 0), (1 << 30, 2, 1, 0), (1 << 31, 1, 8, 0),
    (BIG, 1, 1, (1 << 31)), (1 << 20, 8, 1 << 62, 1 << 30), (1, 1, (1 << 63) - 1, 128), (3, 2, 4, 512), (-1, 2, 4, 0), (3, 2, -1, 0)])
def test_rows_of_any_sizes(T, picks, experts, rows):
    assert mx.expert_rows(T, picks, experts) == rows
    assert mx.expert_plan_workspace_bytes(T, picks, experts) >= 0


def test_too_many_choices_are_refused():
    A = [0x10000 * (i + 1) for i in range(6)]  # aligned addresses, never read
    for T, picks in ((BIG, BIG), (BIG, 2), (1 << 30, 2), (BIG, 1)):
        assert mx.lib().mx_expert_plan(A[0], 4, T, picks, 512, A[1], A[2], A[3], A[4], A[5], 1 << 40, None) == 2, (T, picks)
