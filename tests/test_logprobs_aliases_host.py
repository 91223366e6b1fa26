"""Gradients over the logits: rows that begin inside the logits' own, where
workgroups would read what others write, are refused.  No GPU needed: every call
here is."""
import pytest

import ternary_weight_absmean_amd as bl
from test_block_host import BL_ERR_ALIGN, BL_ERR_SHAPE

lib = bl.library()
AT = 1 << 24


def call(dx, m=3, n=1000, stride=1200, kind=0, lse=1 << 20):
    return lib.bl_logprobs_backward(AT, kind, m, n, stride, 1.0, None, lse, None, None, None, 1 << 20, dx, stride, None)


@pytest.mark.parametrize("kind,size", [(0, 2), (1, 4)])
@pytest.mark.parametrize("m,n,stride", [(3, 1000, 1200), (1, 1000, 1000), (1, 7, 9), (2, 1, 1), (5, 64, 64), (1000, 100, 300)])
def test_rows_that_cross_are_refused(m, n, stride, kind, size):
    rows = [range(r * stride, r * stride + n) for r in range(m)]
    inside = set(e for r in rows for e in r)
    for apart in sorted({1, n // 2, n - 1, n, stride - n, stride - 1, stride, stride + 1, (m - 1) * stride, (m - 1) * stride + n - 1,
                         (m - 1) * stride + n, m * stride, m * stride + n}):
        if apart <= 0:
            continue
        for side in (1, -1):
            crosses = any(side * apart + e in inside for r in rows for e in (r[0], r[-1]))
            crosses = crosses or any(e - side * apart in inside for r in rows for e in (r[0], r[-1]))
            if crosses:
                assert call(AT + side * apart * size, m, n, stride, kind) == BL_ERR_SHAPE, (apart, side)


def test_what_is_wrong_otherwise_is_said_first():
    assert call(AT + 1) == BL_ERR_ALIGN and call(AT + 2, lse=(1 << 20) + 2) == BL_ERR_ALIGN
