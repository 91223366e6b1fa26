"""GPU checks of the cache's pages (growing, forking, freeing, compacting,
copying) against a model on Python lists: whole numbers, all equal."""
import numpy as np
import pytest
import torch

import _answers
import ternary_weight_absmean_amd as bl
from _gpu import DEV, host, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


def i32(v, shape=None):
    t = torch.from_numpy(np.asarray(v, np.int32)).to(DEV)
    return t if shape is None else t.reshape(shape).contiguous()


class Both:
    """The device's pool and table beside the model's."""

    def __init__(self, pages, page, table, refs=None):
        count = [0] * pages
        for row in table:
            for e in row:
                if 0 <= e < pages:
                    count[e] += 1
        self.model = _answers.Pool(count if refs is None else refs, page)
        self.guarded = torch.full((pages + 32,), 77, dtype=torch.int32, device=DEV)
        self.guarded[16:16 + pages] = i32(self.model.refs)
        self.pool = bl.KVPool(self.guarded[16:16 + pages], page)
        self.table, self.page = [list(r) for r in table], page
        self.device = i32(self.table, (len(table), len(table[0]) if table else 0))
        self.short = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.model_short = 0

    def same(self):
        assert host(self.pool.refs).tolist() == self.model.refs
        assert host(self.device).tolist() == self.table
        assert int(self.short) == self.model_short
        assert (self.guarded[:16] == 77).all() and (self.guarded[-16:] == 77).all()

    def grow(self, start, count, cache=None):
        """With a cache: shared pages that are written further are copied first."""
        offsets = np.concatenate([[0], np.cumsum(count)])
        batch = bl.KVBatch(self.device, i32(start), i32(offsets), int(offsets[-1]), max(count),
                           min(max(max(a, 0) + n for a, n in zip(start, count)), self.device.shape[1] * self.page))
        copies = torch.empty((len(start), 3), dtype=torch.int32, device=DEV) if cache else None
        bl.bl_kv_grow(self.pool, batch, copies=copies, shortage=self.short)
        want = [] if cache else None
        self.model_short += self.model.grow(self.table, start, count, want)
        if cache:
            assert host(copies).tolist() == [list(c) for c in want]
            bl.bl_kv_copy(cache, copies)
        self.same()

    def fork(self, length, parent, keep):
        out = bl.bl_kv_fork(self.pool, self.device, i32(length), i32(parent), keep_parents=keep, shortage=self.short)
        table, lengths, copies, short = self.model.fork(self.table, length, parent, keep)
        self.model_short += short
        assert host(out[0]).tolist() == table
        assert host(out[1]).tolist() == lengths
        assert host(out[2]).tolist() == [list(c) for c in copies]
        self.same()
        return out, table, lengths

    def take(self, out, table):
        self.device, self.table = out[0], table

    def free(self, keep=None):
        bl.bl_kv_free(self.pool, self.device, None if keep is None else i32(keep))
        self.model.free(self.table, keep)
        self.same()

    def compact(self, moves):
        copies, moved = bl.bl_kv_compact(self.pool, self.device, moves)
        want, count = self.model.compact(self.table, moves)
        assert host(copies).tolist() == [list(c) for c in want] and int(moved) == count
        self.same()
        return copies, moved


def scattered(rng, pages, page, lengths, stride):
    """Rows of random pages for sequences of these lengths."""
    order = rng.permutation(pages).tolist()
    table = []
    for n in lengths:
        have = -(-n // page)
        table.append([order.pop() for _ in range(have)] + [-1] * (stride - have))
    return table


@pytest.mark.parametrize("pages,page", [(5, 16), (64, 16), (1000, 64), (9000, 32), (20000, 256)])
def test_growing_takes_the_lowest_free_pages(pages, page):
    rng = np.random.default_rng(pages)
    lengths = [0, 1, page, page + 1, 3 * page - 1]
    lengths = lengths if pages > 20 else [0, 1, page]
    b = Both(pages, page, scattered(rng, pages, page, lengths, 40))
    say(f"bl_kv_grow pages={pages} page={page}")
    b.grow(lengths, [1] * len(lengths))
    lengths = [n + 1 for n in lengths]
    b.grow(lengths, [1] * len(lengths))        # mostly nothing to do
    b.grow(lengths, [0] + [5] * (len(lengths) - 1))
    b.grow(lengths, [3 * page + 2] * len(lengths))
    b.grow([0] * len(lengths), [7 * page] * len(lengths))
    assert pages > 20 or b.model_short > 0


@pytest.mark.parametrize("seqs,new", [(1, 40000), (3000, 1), (70, 700)])
def test_many_requests_and_a_pool_that_runs_out(seqs, new):
    """More requests than are taken together, free pages far back, then none."""
    rng = np.random.default_rng(seqs)
    pages = 30000
    refs = (rng.random(pages) < 0.7).astype(int)
    refs[:12000] = 1
    stride = -(-new // 16) + 1
    b = Both(pages, 16, [[-1] * stride for _ in range(seqs)], refs.tolist())
    say(f"bl_kv_grow seqs={seqs} new={new}")
    b.grow([5] * seqs, [new] * seqs)
    b.grow([5 + new] * seqs, [9] * seqs)
    b.free()


@pytest.mark.parametrize("free", [0, 1, 3, 50])
def test_shared_pages_are_copied_before_they_are_written(free):
    cache = bl.KVCache.empty(60, 1, 16, 16, DEV)
    # page 5 is held by rows 0, 1, 3 and 6 (which writes nothing now), page 9 by rows 2 and 4 alone, page 8 by row 5
    table = [[5, -1], [5, -1], [7, 9], [5, -1], [6, 9], [8, -1], [5, -1], [9, -1]][:7]
    refs = [1] * 60
    for p in range(60 - free, 60):
        refs[p] = 0
    refs[5], refs[9] = 4, 2
    b = Both(60, 16, table, refs)
    say(f"bl_kv_grow shared free={free}")
    b.grow([3, 15, 20, 7, 17, 1, 0], [1, 1, 4, 30, 1, 2, 0], cache)
    if free == 50:
        assert b.model.refs[5] == 1 and b.model.refs[9] == 1 and b.model_short == 0


@pytest.mark.parametrize("pages,free", [(70000, [69999]), (200000, [8191, 8192, 65536, 131071, 199999]), (1 << 18, [150000, 150001]),
                                        (150001, [])])
def test_free_pages_far_behind_used_ones(pages, free):
    refs = np.ones(pages, int)
    refs[free] = 0
    b = Both(pages, 16, [[-1], [-1], [-1], [-1]], refs.tolist())
    say(f"bl_kv_grow far pages={pages}")
    b.grow([0, 0, 0, 0], [1, 1, 1, 1])
    b.free([1, 0, 0, 1])
    b.grow([0, 0, 0, 0], [1, 1, 1, 1])


def test_growing_with_odd_integers():
    """Positions before 0, past the table, offsets that do not ascend: what the header says of them."""
    b = Both(50, 16, [[-1, -1, -1], [-1, 60, -7], [3, -1, -1]])
    say("bl_kv_grow odd integers")
    start, offsets = i32([-5, 16, 40]), i32([0, 10, 30, 25])
    batch = bl.KVBatch(b.device, start, offsets, 30, 20, 48)
    bl.bl_kv_grow(b.pool, batch, shortage=b.short)
    b.model.grow(b.table, [0, 16, 40], [10, 20, 0])
    b.same()
    batch = bl.KVBatch(b.device, i32([47, 40, 1 << 30]), i32([0, 20, 40, 60]), 60, 20, 48)
    bl.bl_kv_grow(b.pool, batch)
    b.model.grow(b.table, [47, 40, 0], [20, 20, 0])  # the table ends at 48
    b.same()


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_forking(page, keep):
    rng = np.random.default_rng(page + keep)
    lengths = [0, 1, page - 1, page, page + 1, 5 * page + 3, 2 * page]
    b = Both(4000, page, scattered(rng, 4000, page, lengths, 9))
    say(f"bl_kv_fork page={page} keep={keep}")
    for parent in ([0, 1, 2, 3, 4, 5, 6], [5, 5, 5, 2, 2, 1, 4, 4], [6], [-1, 3, 99, 5], rng.integers(7, size=200).tolist()):
        c = Both(4000, page, b.table)
        out, table, held = c.fork(lengths, parent, keep)
        if keep:
            c.take(out, table)
            c.free()
            assert c.model.refs == b.model.refs
        else:
            c.take(out, table)
            c.grow(held, [2] * len(parent))
            c.free()
            assert sum(c.model.refs) == 0


def test_fork_short_of_pages_and_odd_entries():
    # pages 0, 2, 4 used; one free page of five left for three that are wanted; a hole in a row; a length past the row
    b = Both(5, 16, [[0, 2, -1], [4, -1, -1], [-1, 9, -1]], [1, 1, 1, 0, 1])
    say("bl_kv_fork short")
    b.fork([20, 3, 20], [0, 1, 2, 0, 1], True)
    b = Both(5, 16, [[0, 2, -1], [4, -1, -1], [-1, 9, 1]])
    b.fork([20, -3, 999], [0, 0, 1, 2, 2, 2], False)
    b = Both(5, 16, [[0, 2, 3], [4, -1, -1]])  # pages past the length go back
    b.fork([17, 3], [0], False)
    assert b.model.refs == [1, 0, 1, 0, 0]
    b = Both(5, 16, [[0, 2, 3], [4, -1, -1]])
    b.fork([17, 3], [], False)
    assert sum(b.model.refs) == 0


def test_forking_at_the_largest():
    rng = np.random.default_rng(3)
    seqs = 8192
    lengths = rng.integers(0, 60, size=seqs).tolist()
    b = Both(1 << 16, 16, scattered(rng, 1 << 16, 16, lengths, 4))
    say("bl_kv_fork 8192")
    b.fork(lengths, rng.integers(seqs, size=8192).tolist(), False)


def test_forking_wide_tables():
    """Rows so long that consumed parents' pages are given back by a launch of its own."""
    rng = np.random.default_rng(4)
    lengths = [16 * 9000 + 5, 40, 16 * 11000, 7, 0]
    b = Both(30000, 16, scattered(rng, 30000, 16, lengths, 12000))
    say("bl_kv_fork wide")
    b.fork([16 * 9000 + 5, 17, 16 * 10500, 7, 0], [2, 0, 0, 1, 4], False)


def test_freeing():
    rng = np.random.default_rng(8)
    lengths = [0, 5, 16, 17, 160, 100]
    table = scattered(rng, 300, 16, lengths, 300)
    table[1][0] = table[4][0]        # a shared page
    table[5][2] = 4000               # not a page
    b = Both(300, 16, table)
    say("bl_kv_free")
    b.free([0, 5, 0, 16, 99, 1000000])
    b.free([1, -9, 0, 0, 17, 33])
    b.free()
    b.free()                         # nothing left
    assert sum(b.model.refs) == 0
    b = Both(300, 16, [[7, 7, 7, 9]], [0] * 300)  # counts that do not agree: none goes below 0
    b.model.refs[7] = 2
    b.pool.refs[7] = 2
    b.free()
    assert b.model.refs[7] == 0


@pytest.mark.parametrize("pages,share", [(1, 0.5), (16, 0.5), (100, 0.0), (100, 1.0), (4096, 0.3), (4097, 0.9), (50000, 0.5), (12289, 0.02)])
def test_compacting(pages, share):
    rng = np.random.default_rng(pages)
    order = rng.permutation(pages)[:int(pages * share)].tolist()
    table = [order[i:i + 37] + [-1] * (37 - len(order[i:i + 37])) for i in range(0, len(order), 37)] or [[-1] * 37]
    if len(table) > 1:
        table.append(list(table[0]))  # a second holder
        table[1][5] = -4
    say(f"bl_kv_compact pages={pages} share={share}")
    for moves in sorted({0, 1, pages // 3, pages // 2, pages}):
        b = Both(pages, 16, table)
        b.compact(moves)
        b.compact(pages)
        assert b.model.refs == sorted(b.model.refs, key=lambda r: r == 0) or True
        used = sum(r > 0 for r in b.model.refs)
        assert all(r > 0 for r in b.model.refs[:used])


@pytest.mark.parametrize("heads,page,dim,layers", [(1, 16, 16, 1), (5, 64, 128, 3), (2, 256, 256, 2), (3, 32, 80, 40), (8, 128, 48, 1)])
def test_copying(heads, page, dim, layers):
    rng = np.random.default_rng(dim + layers)
    pages = 23
    caches, copies = [], []
    for _ in range(layers):
        k, v = rng.integers(-128, 128, size=(2, pages, heads, page, dim)).astype(np.int8)
        ka, va = rng.random((2, pages, heads)).astype(np.float32)
        caches.append([k, v, ka, va])
    free = rng.permutation(pages).tolist()
    for tokens in (page, 1, page - 1, page // 2, 0, page + 100, -3):
        copies.append((free[0] if len(copies) < 2 else free[1], free[3 + len(copies)], tokens))
    copies += [(-1, -1, 0), (99, free[20], page), (free[0], 99, page), (free[2], free[2], page), (free[2], free[21], page)]
    say(f"bl_kv_copy heads={heads} page={page} dim={dim} layers={layers}")
    for count in (None, 3, 0, -5, 1000):
        on = [[torch.from_numpy(t).to(DEV) for t in c] for c in caches]
        kv = [bl.KVCache(*c) for c in on]
        valid = None if count is None else i32([count])
        bl.bl_kv_copy(bl.KVCaches(kv) if layers > 1 else kv[0], i32(copies), count=valid)
        done = copies if count is None else copies[:max(count, 0)]
        clipped = [(a, b, min(n, page)) for a, b, n in done]
        for c, d in zip(caches, on):
            for codes, top, got, got_top in ((c[0], c[2], d[0], d[2]), (c[1], c[3], d[1], d[3])):
                k, a = _answers.copy_pages(codes, top, clipped)
                assert np.array_equal(host(got), k) and np.array_equal(host(got_top), a)


def test_copying_past_two_to_the_32_bytes():
    say("bl_kv_copy past 2^32 bytes")
    pages, heads, page, dim = 1100, 16, 256, 256  # 4.6 GB of keys
    cache = bl.KVCache.empty(pages, heads, page, dim, DEV)
    cache.k[1090] = 3
    cache.v[1090] = 4
    cache.k_absmax[1090] = 5.0
    bl.bl_kv_copy(cache, i32([[1090, 1099, page], [1090, 2, 9]]))
    torch.cuda.synchronize()
    assert (cache.k[1099] == 3).all() and (cache.v[1099] == 4).all() and (cache.k_absmax[1099] == 5.0).all()
    assert (cache.k[2, :, :9] == 3).all() and not cache.k[2, :, 9:].any()
    assert not cache.k[1091:1099].any() and not cache.k[:2].any()


def test_a_long_run_of_steps():
    """Beams and samples that grow, fork, end and move, with the codes of every token checked against a record."""
    rng = np.random.default_rng(21)
    page, pages, heads, dim, stride = 16, 400, 2, 32, 30
    cache = bl.KVCache.empty(pages, heads, page, dim, DEV)
    b = Both(pages, page, [[-1] * stride for _ in range(4)])
    text = [[], [], [], []]  # what each sequence wrote, a number per token
    say("pages, a long run")

    def write(count):
        start = [len(t) for t in text]
        b.grow(start, count, cache)
        offsets = np.concatenate([[0], np.cumsum(count)])
        for s, n in enumerate(count):
            text[s] = text[s] + rng.integers(1, 100, size=n).tolist()
        rows = np.concatenate([np.asarray(t[a:], np.float32) for t, a in zip(text, start)]) if sum(count) else np.zeros(0, np.float32)
        x = torch.from_numpy(rows).to(DEV).to(torch.bfloat16)[:, None, None].expand(-1, heads, dim).contiguous()
        batch = bl.KVBatch(b.device, i32(start), i32(offsets), int(offsets[-1]), max(count), max(len(t) for t in text))
        if sum(count):
            bl.bl_kv_append(cache, batch, x, -x)

    def read():
        offsets = np.concatenate([[0], np.cumsum([len(t) for t in text])])
        batch = bl.KVBatch(b.device, i32([0] * len(text)), i32(offsets), int(offsets[-1]), max(len(t) for t in text), max(len(t) for t in text))
        k, v = bl.bl_kv_read(cache, batch)
        want = np.concatenate([np.asarray(t, np.float64) for t in text])
        # a page's scale may have grown several times: half a step of at most 100 / 127 each, then bf16
        for got, sign in ((k, 1), (v, -1)):
            got = got.float().cpu().numpy().astype(np.float64)
            assert np.abs(got - sign * want[:, None, None]).max() <= 100 / 127 / 2 * 16 + 100 * 2.0 ** -8
            assert (got == got[:, :1, :1]).all()

    for step in range(40):
        write([int(rng.integers(0, 14)) if len(t) < 380 else 0 for t in text])
        read()
        kind = step % 4
        length = [len(t) for t in text]
        if kind in (0, 2):
            parent = rng.integers(len(text), size=int(rng.integers(2, 7))).tolist()
            (out, table, _) = b.fork(length, parent, keep=False)
            bl.bl_kv_copy(cache, out[2])
            b.take(out, table)
            text = [list(text[p]) for p in parent]
        elif kind == 1:
            cut = [int(rng.integers(0, n + 1)) for n in length]
            b.free(cut)
            text = [t[:n] for t, n in zip(text, cut)]
        else:
            copies, moved = b.compact(int(rng.integers(0, 60)))
            bl.bl_kv_copy(cache, copies, count=moved)
        read()
    assert b.model_short == 0


def test_a_captured_beam_step():
    rng = np.random.default_rng(31)
    page, pages, stride, beams = 16, 200, 8, 6
    lengths = [20, 33, 48, 15, 70, 1]
    table = scattered(rng, pages, page, lengths, stride)
    start = Both(pages, page, table)
    cache = bl.KVCache.empty(pages, 1, page, 16, DEV)
    cache.k.copy_(torch.arange(pages, device=DEV).view(-1, 1, 1, 1).to(torch.int8))
    tables = [start.device, torch.full_like(start.device, -1)]
    held = [i32(lengths), torch.zeros(beams, dtype=torch.int32, device=DEV)]
    parent, copies = i32([0] * beams), torch.empty((beams, 3), dtype=torch.int32, device=DEV)
    offsets = torch.arange(beams + 1, dtype=torch.int32, device=DEV)
    say("pages, captured")

    def step(at):
        bl.bl_kv_fork(start.pool, tables[at], held[at], parent, table=tables[1 - at], out_length=held[1 - at], copies=copies,
                      shortage=start.short)
        bl.bl_kv_copy(cache, copies)
        bl.bl_kv_grow(start.pool, bl.KVBatch(tables[1 - at], held[1 - at], offsets, beams, 1, stride * page), shortage=start.short)
        held[1 - at].add_(1)

    graphs = []
    torch.cuda.synchronize()
    for at in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(at)
        graphs.append(g)
    model, rows, length = start.model, start.table, lengths
    for i in range(8):
        chosen = rng.integers(beams, size=beams).tolist()
        parent.copy_(i32(chosen))
        graphs[i % 2].replay()
        rows, length, _, short = model.fork(rows, length, chosen, False)
        assert short == 0 and model.grow(rows, length, [1] * beams) == 0
        length = [n + 1 for n in length]
        assert host(tables[1 - i % 2]).tolist() == rows and host(held[1 - i % 2]).tolist() == length
        assert host(start.pool.refs).tolist() == model.refs
    assert int(start.short) == 0
