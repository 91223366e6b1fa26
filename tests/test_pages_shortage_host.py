"""The reference for growing with copies when pages run out, against what the
header says of it.  No GPU needed."""
import numpy as np
import pytest

import _answers


@pytest.mark.parametrize("start", [(20, 17), (17, 20)])
def test_sharers_of_a_page_without_a_free_one(start):
    """Neither of two writers of a page may write while both hold it; with one page free, one is copied."""
    pool = _answers.Pool([1] * 9 + [2], 16)
    table, copies = [[0, 9], [1, 9]], []
    assert pool.grow(table, start, [1, 1], copies) == 2
    assert copies == [(9, -1, 0), (9, -1, 0)] and pool.refs[9] == 2 and table == [[0, 9], [1, 9]]
    pool.refs[4] = 0
    copies = []
    assert pool.grow(table, start, [1, 1], copies) == 0
    assert copies == [(9, 4, start[0] % 16), (-1, -1, 0)] and pool.refs[9] == 1 and table == [[0, 4], [1, 9]]


@pytest.mark.parametrize("seed", range(20))
def test_a_sequence_that_may_write_holds_its_page_alone(seed):
    """Whatever is free: a page that is written has one holder, or its copies entry says that it must not be."""
    rng = np.random.default_rng(seed)
    seqs, pages, page = 30, 40, 16
    table = [[int(e)] for e in rng.integers(8, size=seqs)]
    refs = [0] * pages
    for row in table:
        refs[row[0]] += 1
    refs[8:] = (rng.random(pages - 8) < 0.5 + 0.5 * (seed % 2)).astype(int).tolist()
    pool, copies = _answers.Pool(refs, page), []
    start, count = rng.integers(1, 12, size=seqs).tolist(), (rng.random(seqs) < 0.8).astype(int).tolist()
    before = sum(refs)
    short = pool.grow(table, start, count, copies)
    assert sum(pool.refs) == before and short == sum(a >= 0 and b < 0 for a, b, _ in copies)
    for row, n, (a, b, _) in zip(table, count, copies):
        assert n == 0 or (pool.refs[row[0]] > 1) == (a >= 0 and b < 0)
