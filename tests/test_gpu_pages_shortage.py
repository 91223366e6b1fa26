"""GPU checks of growing with copies: many writers of one page, and pages that
run out.  Whole numbers, all equal to the model's or to those written here."""
import numpy as np
import pytest
import torch

import ternary_weight_absmean_amd as bl
from _gpu import DEV, host, say
from test_gpu_pages import Both, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


@pytest.mark.parametrize("start", [(20, 17), (17, 20)])
def test_sharers_of_a_page_without_a_free_one(start):
    """Neither of two writers of a page may write while both hold it; with one page free, one is copied."""
    refs = i32([1] * 9 + [2])
    table = i32([[0, 9], [1, 9]])
    pool, short = bl.KVPool(refs, 16), torch.zeros(1, dtype=torch.int32, device=DEV)
    batch = bl.KVBatch(table, i32(start), i32([0, 1, 2]), 2, 1, 32)
    copies = torch.full((2, 3), 7, dtype=torch.int32, device=DEV)
    say(f"bl_kv_grow two sharers start={start}")
    bl.bl_kv_grow(pool, batch, copies=copies, shortage=short)
    assert host(copies).tolist() == [[9, -1, 0], [9, -1, 0]] and int(short) == 2
    assert host(refs).tolist() == [1] * 9 + [2] and host(table).tolist() == [[0, 9], [1, 9]]
    cache = bl.KVCache.empty(10, 1, 16, 16, DEV)
    cache.k[9] = 3
    keep = cache.k.clone()
    bl.bl_kv_copy(cache, copies)
    assert torch.equal(cache.k, keep)
    refs[4] = 0
    bl.bl_kv_grow(pool, batch, copies=copies, shortage=short)
    assert host(copies).tolist() == [[9, 4, start[0] % 16], [-1, -1, 0]] and int(short) == 2
    assert host(refs).tolist() == [1] * 10 and host(table).tolist() == [[0, 4], [1, 9]]


@pytest.mark.parametrize("seqs,free,outside", [(8192, 9000, 0), (8192, 8191, 0), (8192, 8190, 0), (8192, 3000, 2), (1025, 1025, 1),
                                               (1024, 0, 0), (64, 63, 0), (65, 64, 1)])
def test_many_sequences_write_on_in_one_page(seqs, free, outside):
    rng = np.random.default_rng(seqs + free)
    pages = seqs + free + 10
    refs = np.ones(pages, int)
    refs[rng.permutation(np.arange(10, pages))[:free]] = 0
    refs[5] = seqs + outside
    b = Both(pages, 16, [[5, -1] for _ in range(seqs)], refs.tolist())
    cache = bl.KVCache.empty(pages, 1, 16, 16, DEV)
    say(f"bl_kv_grow {seqs} writers of one page, {free} free")
    b.grow(rng.integers(1, 16, size=seqs).tolist(), [1] * seqs, cache)
    assert b.model_short == max(0, seqs - (free if outside else max(free, 0) + (free >= seqs - 1)))


@pytest.mark.parametrize("seqs,shared,free", [(8192, 4096, 4000), (8192, 8192, 3000), (3000, 40, 1500), (700, 3, 400), (130, 60, 500)])
def test_sharers_and_new_pages_among_each_other(seqs, shared, free):
    """Pages of several writers, of writers and of sequences that wait, rows without a page, further pages."""
    rng = np.random.default_rng(seqs + shared)
    pages = shared + free + 50
    table, refs = [], np.ones(pages, int)
    refs[:shared] = 0
    for s in range(seqs):
        e = int(rng.integers(shared)) if shared < seqs else s % shared
        if rng.random() < 0.05:
            e = -1
        else:
            refs[e] += 1
        table.append([e, -1, -1])
    refs[:shared] += rng.random(shared) < 0.3  # held by rows that are not of the batch
    refs[shared + rng.permutation(pages - shared)[:free]] = 0
    b = Both(pages, 16, table, refs.tolist())
    cache = bl.KVCache.empty(pages, 1, 16, 16, DEV)
    say(f"bl_kv_grow sharers seqs={seqs} pages={shared} free={free}")
    start = rng.integers(0, 17, size=seqs).tolist()
    count = (rng.integers(0, 30, size=seqs) * (rng.random(seqs) < 0.5)).tolist()
    b.grow(start, count, cache)
    b.free(rng.integers(0, 3, size=seqs).tolist())
    b.grow(start, [1] * seqs, cache)
