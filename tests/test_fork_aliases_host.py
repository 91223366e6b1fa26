"""Forks whose outputs lie in what other workgroups still read are refused before
anything is enqueued.  No GPU needed."""
import pytest

import ternary_weight_absmean_amd as bl
from test_answers_host import pool
from test_block_host import BL_ERR_NULL, BL_ERR_SHAPE

lib = bl.library()
SEQS, CHILDREN, STRIDE, PAGES = 5, 7, 4, 100
SIZES = dict(table=SEQS * STRIDE, length=SEQS, parent=CHILDREN, out=CHILDREN * STRIDE, out_length=CHILDREN, copies=3 * CHILDREN,
             refs=PAGES, shortage=1)
APART = {name: (i + 1) << 16 for i, name in enumerate(SIZES)}


def call(**kw):
    at = dict(APART, **kw)
    keep, pp = pool(at["refs"], PAGES, 16)
    return lib.bl_kv_fork(pp, at["table"], STRIDE, at["length"], SEQS, at["parent"], CHILDREN, 0, at["out"], at["out_length"],
                          at["copies"], at["shortage"], None)


@pytest.mark.parametrize("out", ["out", "out_length", "copies"])
@pytest.mark.parametrize("other", list(SIZES))
def test_outputs_share_no_element(out, other):
    if out == other:
        return
    first, size = APART[other], SIZES[other]
    for at in (first, first + 4 * (size - 1), first - 4 * (SIZES[out] - 1)):
        assert call(**{out: at}) == BL_ERR_SHAPE, (out, other, at - first)
    # next to each other they are taken (as far as what is missing here)
    for at in (first + 4 * size, first - 4 * SIZES[out]):
        assert call(**{out: at, "parent" if other != "parent" else "table": None}) == BL_ERR_NULL
