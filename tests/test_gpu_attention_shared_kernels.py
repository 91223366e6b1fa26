"""GPU checks of the attention over shared prefixes on the kernels that take the
prefixes together, at small and odd sizes: max_prefix and max_len are bounds, and
with large ones the rule decides for these kernels whatever the batch holds.
Every case asserts that it does."""
import functools

import numpy as np
import pytest
import torch

import _block
import test_gpu_attention_shared as base
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, host, say
from test_block_host import cache_batch, struct, FAKE
from test_gpu_attention_shared import Answers, check
from test_gpu_device_integers import Walled
from test_gpu_kv_cache import heads, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

lib = bl.library()


def shares(n_heads, q_heads, dim, page, seqs, tokens, max_new, max_len, groups, max_group, max_prefix):
    """Whether these bounds have the prefixes taken together."""
    (c, cp), (b, bp) = cache_batch(pages=1 << 16, heads=n_heads, page=page, dim=dim, seqs=seqs, tokens=tokens, max_new=max_new,
                                   max_len=max_len, stride=-(-max_len // page))
    s, sp = struct(bl.KVShared, FAKE, FAKE, groups, max_group, max_prefix)
    return lib.bl_attention_shared_workspace_bytes(cp, bp, sp, q_heads) != lib.bl_attention_workspace_bytes(cp, bp, q_heads)


class NotTogether(Exception):
    """No such bounds have the prefixes taken together."""


class Far(Answers):
    """A batch whose bounds are the smallest powers of two (times up to `times`) that have its prefixes taken together;
    the table has entries without a page for the rest of them.  `extra`: further room behind the longest prefix."""

    def __init__(self, rng, groups, n_heads, dim, page, q_heads, times=1, extra=0):
        super().__init__(rng, groups, n_heads, dim, page)
        longest = int((self.start + np.diff(self.offsets)).max())
        sizes = (n_heads, q_heads, dim, page, len(self.start), self.total, max(self.new))
        self.max_prefix = 64
        while self.max_prefix < max(self.prefix) or not self.taken(sizes, longest + extra):
            self.max_prefix *= 2
            if self.max_prefix >= 1 << 23:
                raise NotTogether
        least = self.max_prefix
        for more in range(times, 0, -1):
            self.max_prefix = least * more
            if self.taken(sizes, longest + extra):
                break
        self.max_len = self.max_prefix + longest + extra

    def taken(self, sizes, room):
        return shares(*sizes, self.max_prefix + room, len(self.prefix), max(self.width), self.max_prefix)

    def wide(self):
        table = np.full((len(self.start), -(-self.max_len // self.page)), -1)
        table[:, :self.table.shape[1]] = self.table
        return i32(table)

    def step(self, start, offsets):
        return bl.KVBatch(self.wide(), i32(start), i32(offsets), int(offsets[-1]), max(self.new), self.max_len)

    def shared(self):
        return super().shared(self.max_prefix)


BOUNDS = [dict(), dict(times=4), dict(extra=5000), dict(times=2, extra=300), dict(times=4, extra=9000), dict(times=16, extra=2500)]


@pytest.mark.parametrize("n_heads,q_heads,dim,page", base.GEOMETRY)
@pytest.mark.parametrize("groups", base.GROUPS)
def test_matches_reference(n_heads, q_heads, dim, page, groups):
    rng = np.random.default_rng(dim + q_heads + len(groups))
    q = None
    for bounds in BOUNDS:
        try:
            c = Far(np.random.default_rng(dim + q_heads), groups, n_heads, dim, page, q_heads, **bounds)
        except NotTogether:
            assert bounds.get("extra")  # much room behind the prefixes may be for the other kernels
            continue
        q = heads(rng, c.total, q_heads, dim) if q is None else q
        say(f"bl_attention_shared groups={groups} heads={n_heads}/{q_heads} dim={dim} page={page} bounds={c.max_prefix}, {c.max_len}")
        check(c, q)


def drawn(seed):
    """A batch of any of the sizes that share, its sequences well inside the bounds."""
    rng = np.random.default_rng(seed)
    pick = lambda *v: v[int(rng.integers(len(v)))]  # noqa: E731
    log = lambda top: int(2 ** rng.uniform(0, np.log2(top)))  # noqa: E731
    for _ in range(10000):
        n_heads, dim, page = pick(1, 1, 2, 3, 4, 8), 16 * int(rng.integers(1, 17)), pick(16, 32, 64, 128, 256)
        q_heads = n_heads * pick(1, 2, 4, 5, 8, 16, 20)
        new = log((4, 40, 200)[seed % 3])
        groups = []
        for _ in range(pick(1, 1, 1, 2, 3, 8)):
            width = log(60)
            prefix = pick(0, 63, 64, 65, log(1500), 64 * log(24), log(1500))
            groups.append((prefix, [pick(0, 1, log(500), 64 * log(8)) for _ in range(width)], [1 + int(rng.integers(new)) for _ in range(width)]))
        total = sum(sum(n) for _, _, n in groups)
        cost = sum((p + a + n) * n for p, rest, each in groups for a, n in zip(rest, each)) * q_heads * dim
        if cost > 2.5e9 or total > 5000:
            continue
        room = log(16000)
        most = max(p for p, _, _ in groups)
        max_prefix = max(64 * log(2048), most)
        longest = max(p + a + n for p, rest, each in groups for a, n in zip(rest, each))
        widths = [len(r) for _, r, _ in groups]
        if shares(n_heads, q_heads, dim, page, sum(widths), total, max(n for _, _, e in groups for n in e), max(max_prefix + room, longest),
                  len(groups), max(widths), max_prefix):
            c = Answers(rng, groups, n_heads, dim, page)
            c.__class__ = Far
            c.max_prefix, c.max_len = max_prefix, max(max_prefix + room, longest)
            return rng, c, q_heads
    raise AssertionError("nothing drawn")


@pytest.mark.parametrize("seed", range(120))
def test_drawn_batches(seed):
    rng, c, q_heads = drawn(seed)
    say(f"bl_attention_shared drawn seed={seed} prefix={c.prefix} width={c.width} heads={c.k.shape[1]}/{q_heads} dim={c.k.shape[3]} "
        f"page={c.page} total={c.total} bounds={c.max_prefix}, {c.max_len}")
    check(c, heads(rng, c.total, q_heads, c.k.shape[3]))


# the checks of small batches, on bounds that have them taken together
SAME = [(base.test_missing_pages_and_rows_that_see_nothing, 4, {}), (base.test_nan_stays_with_those_that_see_it, 2, {}),
        (base.test_what_is_not_visible_does_not_matter, 4, {}), (base.test_sharp_and_flat_softmax_and_scales_far_apart, 4, dict(width=1)),
        (base.test_sharp_and_flat_softmax_and_scales_far_apart, 4, dict(width=30)),
        (base.test_strided_queries_another_stream_and_a_graph, 4, {})]


@pytest.mark.parametrize("times,extra", [(1, 0), (1, 5000), (16, 0)])
@pytest.mark.parametrize("which", range(len(SAME)))
def test_small_batches(which, times, extra, monkeypatch):
    test, q_heads, kw = SAME[which]
    made = []

    def far(*a, **k):
        made.append(Far(*a, q_heads=q_heads, times=times, extra=extra, **k))
        return made[-1]

    monkeypatch.setattr(base, "Answers", far)
    say(f"bl_attention_shared, together, times={times} extra={extra}: {test.__name__}")
    test(**kw)
    assert made


@pytest.mark.parametrize("times,extra", [(1, 0), (1, 5000), (16, 0), (16, 5000)])
def test_device_integers_out_of_bounds_stay_inside_the_buffers(times, extra):
    rng = np.random.default_rng(53)
    c = Far(rng, [(128, [10, 40, 3], [1, 2, 1]), (64, [0, 3], [1, 1])], 2, 64, 16, 4, times, extra)
    cache, batch = c.device()
    q = bf16(_block.bits(heads(rng, c.total, 4, 64)))
    most = c.max_prefix
    say(f"bl_attention_shared odd integers, together, times={times} extra={extra}")
    for group, prefix, start in (([0, 99, -5], [1 << 30, -3], None), ([-7, 2, 5], [most, 640], None), ([3, 1, 5], [0, 64], None),
                                 ([0, 3, 5], [128, 64], [-9, 1 << 30, 0, 5, 64]), ([0, 0, 0], [64, 64], None), ([0, 3, 5], [most, most], None),
                                 ([0, 3, 5], [most, 0], [c.max_len - 1, c.max_len, most, most - 1, -1])):
        shared = bl.KVShared(i32(group), i32(prefix), 3, most)
        b = batch if start is None else bl.KVBatch(batch.page_table, i32(start), batch.offsets, c.total, 2, batch.max_len)
        need = bl.bl_attention_shared_workspace_bytes(cache, b, shared, 4)
        assert need != bl.bl_attention_workspace_bytes(cache, b, 4)
        ws, out, lse = Walled((need,), torch.uint8), Walled(tuple(q.shape), torch.bfloat16), Walled(tuple(q.shape[:2]), torch.float32)
        ws.t.zero_()
        bl.bl_attention_shared(cache, b, shared, q, out=out.t, lse=lse.t, workspace=ws.t)
        torch.cuda.synchronize()
        assert ws.intact() and out.intact() and lse.intact()


@pytest.mark.parametrize("n_heads,q_heads,dim,page,width,prefix,rest", [
    (1, 8, 128, 64, 100, 21500, [3, 190, 250, 700, 1500]), (1, 20, 64, 16, 60, 30000, [0, 255, 256, 900]),
    (1, 8, 256, 32, 90, 24000, [1, 5, 2000]), (2, 16, 80, 64, 40, 27000, [10, 200, 1000])])
def test_rests_that_join_the_prefix_themselves_beside_longer_ones(n_heads, q_heads, dim, page, width, prefix, rest):
    """The prefix in tiles of 128 rows, the rests behind it in several splits: short ones are one split and join the
    prefix's sums themselves, longer ones leave theirs to the join."""
    rng = np.random.default_rng(dim)
    c = Answers(rng, [(prefix, [rest[i % len(rest)] + i % 7 for i in range(width)], [1] * width)], n_heads, dim, page)
    say(f"bl_attention_shared own join and others heads={n_heads}/{q_heads} dim={dim}")
    assert base.together(c, q_heads)
    check(c, heads(rng, c.total, q_heads, dim))


# one token each: the prefix in tiles of 16 rows; 12 tokens of 40 sequences: of 128
@pytest.mark.parametrize("seqs,new", [(12, 1), (40, 12)])
def test_cache_past_two_to_the_32_bytes(seqs, new):
    pages, n_heads, page, dim, q_heads, shared_pages = 70000, 4, 64, 256, 8, 80
    say(f"bl_attention_shared past 2^32 bytes seqs={seqs} new={new}")
    assert (pages - 2000) * n_heads * page * dim > 1 << 32
    rng = np.random.default_rng(seqs)
    used = shared_pages + 2 * seqs
    # a small cache holds the same pages by numbers from 0 on
    k, v = rng.integers(-127, 128, (2, used, n_heads, page, dim)).astype(np.int8)
    ka, va = rng.uniform(0.5, 4, (2, used, n_heads)).astype(np.float32)
    table = np.asarray([list(range(shared_pages)) + [shared_pages + 2 * s, shared_pages + 2 * s + 1] for s in range(seqs)])
    prefix = shared_pages * page
    start = np.asarray([prefix + (11 * s) % 60 for s in range(seqs)])
    offsets = np.arange(seqs + 1) * new
    q = heads(rng, seqs * new, q_heads, dim)
    far = bl.KVCache.empty(pages, n_heads, page, dim, DEV)
    place = pages - 1 - rng.permutation(1900)[:used]  # where page i lies
    where = torch.from_numpy(place).to(DEV)
    for t, a in ((far.k, k), (far.v, v), (far.k_absmax, ka), (far.v_absmax, va)):
        t[where] = torch.from_numpy(a).to(DEV)
    batch = bl.KVBatch(i32(place[table]), i32(start), i32(offsets), seqs * new, new, prefix + 2 * page)
    shared = bl.KVShared(i32([0, seqs]), i32([prefix]), seqs, prefix)
    assert bl.bl_attention_shared_workspace_bytes(far, batch, shared, q_heads) != bl.bl_attention_workspace_bytes(far, batch, q_heads)
    qd = bf16(_block.bits(q))
    got = bl.bl_attention_shared(far, batch, shared, qd)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    near = bl.KVCache(t(k), t(v), t(ka), t(va))
    small = bl.KVBatch(i32(table), i32(start), i32(offsets), seqs * new, new, prefix + 2 * page)
    want, _, bound, _ = _block.attention(q, k, ka, v, va, table, start, offsets, np.float64(np.float32(dim ** -0.5)))
    out = got.float().cpu().numpy().astype(np.float64)
    assert (np.abs(out - want) <= bound + _block.U16 * (np.abs(want) + bound)).all()
    assert torch.equal(got, bl.bl_attention_shared(near, small, shared, qd))
