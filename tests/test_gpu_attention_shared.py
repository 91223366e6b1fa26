"""GPU checks of the attention of sequences that share a prefix against a 64-bit
softmax over each sequence by itself; bounds as derived in _block.attention
(they do not depend on the order of the sums), plus bf16's unit for the
output's rounding."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, host, say
from test_gpu_device_integers import Walled
from test_gpu_kv_cache import Case, heads, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


class Answers(Case):
    """groups: (shared tokens, further tokens of each sequence, new tokens of each)."""

    def __init__(self, rng, groups, n_heads, dim, page):
        self.prefix = [p for p, _, _ in groups]
        self.width = [len(ctx) for _, ctx, _ in groups]
        ctx = [p + a for p, rest, _ in groups for a in rest]
        new = [n for _, _, each in groups for n in each]
        super().__init__(rng, ctx, new, n_heads, dim, page)
        s = 0
        for p, rest, _ in groups:
            for i in range(s + 1, s + len(rest)):
                self.table[i, :p // page] = self.table[s, :p // page]
                if p % page:  # a copy of the page's shared part, as a fork makes it
                    a, b = self.table[s, p // page], self.table[i, p // page]
                    for codes, top in ((self.k, self.ka), (self.v, self.va)):
                        codes[b, :, :p % page] = codes[a, :, :p % page]
                        top[b] = top[a]
            s += len(rest)

    def shared(self, most=None):
        group = np.concatenate([[0], np.cumsum(self.width)])
        return bl.KVShared(i32(group), i32(self.prefix), max(self.width), max(self.prefix) if most is None else most)


def together(c, q_heads, shared=None):
    """Whether the sizes are those for which prefixes are taken together."""
    cache, batch = c.device()
    return bl.bl_attention_shared_workspace_bytes(cache, batch, c.shared() if shared is None else shared, q_heads) != \
        bl.bl_attention_workspace_bytes(cache, batch, q_heads)


def check(c, q, scale=None, q_device=None, shared=None):
    cache, batch = c.device()
    dim = c.k.shape[3]
    scale = dim ** -0.5 if scale is None else scale
    shared = c.shared() if shared is None else shared
    need = bl.bl_attention_shared_workspace_bytes(cache, batch, shared, q.shape[1])
    ws, out, lse = Walled((need,), torch.uint8), Walled(q.shape, torch.bfloat16), Walled(q.shape[:2], torch.float32)
    ws.t.fill_(0xFF)  # NaNs, where read as numbers
    out.t.fill_(9.0)
    lse.t.fill_(9.0)
    qd = bf16(_block.bits(q)) if q_device is None else q_device
    bl.bl_attention_shared(cache, batch, shared, qd, scale=scale, out=out.t, lse=lse.t, workspace=ws.t)
    torch.cuda.synchronize()
    assert ws.intact() and out.intact() and lse.intact()
    want, want_lse, bound, lse_bound = _block.attention(q, c.k, c.ka, c.v, c.va, c.table, c.start, c.offsets,
                                                        np.float64(np.float32(scale)))
    got, got_lse = bf16_bits_to_f64(host(out.t)), host(lse.t).astype(np.float64)
    off = np.abs(got - want) - (bound + _block.U16 * (np.abs(want) + bound))
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} outputs outside their bound, by up to {off.max():.3g}"
    none = np.isinf(want_lse)
    assert (got[none] == 0).all() and (got_lse[none] == -np.inf).all()
    assert (np.abs(got_lse[~none] - want_lse[~none]) <= lse_bound[~none]).all()
    again = bl.bl_attention_shared(cache, batch, shared, qd, scale=scale)
    assert torch.equal(again, out.t)
    return out.t.clone()


GEOMETRY = [  # heads, q heads, dim, page
    (2, 2, 64, 16), (1, 4, 128, 64), (2, 10, 128, 32), (1, 3, 80, 64), (3, 3, 16, 128), (1, 8, 48, 16), (1, 20, 64, 64),
    (2, 4, 256, 64), (1, 2, 144, 32), (1, 1, 192, 256)]
GROUPS = [
    [(64, [0], [1])],
    [(200, [3, 0, 70], [1, 1, 1])],
    [(128, [5] * 9, [1] * 9), (0, [40, 0], [1, 1]), (63, [1, 130], [1, 1])],          # no whole step shared
    [(700, [0, 10, 90, 200], [3, 1, 6, 2]), (256, [64], [4])],
    [(320, [0, 0, 17], [40, 70, 3])],                                               # prompts behind a prefix
    [(192, [1, 2, 3, 4] * 5, [2] * 20), (64, [9, 0], [1, 0])],
]


@pytest.mark.parametrize("n_heads,q_heads,dim,page", GEOMETRY)
@pytest.mark.parametrize("groups", GROUPS)
def test_matches_reference(n_heads, q_heads, dim, page, groups):
    rng = np.random.default_rng(dim + q_heads + len(groups))
    c = Answers(rng, groups, n_heads, dim, page)
    say(f"bl_attention_shared groups={groups} heads={n_heads}/{q_heads} dim={dim} page={page}")
    check(c, heads(rng, c.total, q_heads, dim))


@pytest.mark.parametrize("groups,n_heads,q_heads,dim,page", [
    ([(5000, [20, 300, 0, 77], [1] * 4)], 1, 4, 128, 64),
    ([(20000, [1500, 3], [1, 1]), (64, [9000], [1])], 1, 8, 64, 64),
    ([(4096, [i % 50 for i in range(40)], [1] * 40)], 2, 8, 128, 64),      # many rows of a prefix
    ([(3000, [0, 5, 9], [200, 150, 3])], 1, 4, 128, 16),
    ([(2500, [i for i in range(33)], [2] * 33)], 1, 4, 256, 32),
    ([(1000, [0], [300]), (6400, [0, 1], [1, 5])], 2, 4, 96, 64)])
def test_long_prefixes(groups, n_heads, q_heads, dim, page):
    rng = np.random.default_rng(sum(p for p, _, _ in groups))
    c = Answers(rng, groups, n_heads, dim, page)
    say(f"bl_attention_shared long groups={groups} dim={dim}")
    check(c, heads(rng, c.total, q_heads, dim))


# heads, q heads, dim, page, (prefix, sequences, new tokens each) of one long group, a second beside it
TOGETHER = [
    (1, 4, 64, 16, (20000, 20, 1)), (2, 10, 128, 32, (6000, 16, 1)), (1, 3, 80, 64, (9000, 24, 2)), (3, 3, 16, 128, (9000, 40, 1)),
    (1, 8, 48, 16, (12000, 30, 3)), (1, 20, 64, 64, (20000, 25, 4)), (2, 4, 256, 64, (4000, 16, 1)), (1, 2, 144, 32, (5000, 30, 5)),
    (1, 1, 192, 256, (9000, 25, 1)), (2, 16, 128, 64, (4100, 33, 4)), (2, 8, 64, 64, (9000, 40, 6)), (1, 8, 256, 16, (3000, 60, 4)),
    (2, 4, 128, 64, (9000, 6, 45)), (4, 20, 208, 64, (3000, 6, 70)), (4, 64, 64, 32, (1500, 12, 70)), (4, 64, 112, 64, (1500, 6, 70)),
    (1, 16, 208, 64, (3000, 12, 70)), (1, 16, 208, 16, (6000, 3, 70)), (2, 32, 208, 64, (3000, 3, 70)), (4, 20, 112, 64, (6000, 3, 40)),
    (4, 20, 208, 64, (700, 6, 70)), (4, 64, 64, 16, (700, 12, 70)), (4, 64, 112, 64, (700, 6, 70)), (1, 8, 64, 64, (16000, 24, 9)),
    (1, 8, 128, 64, (12000, 30, 9)), (1, 9, 80, 16, (12000, 30, 8))]


@pytest.mark.parametrize("n_heads,q_heads,dim,page,first", TOGETHER)
def test_prefixes_taken_together(n_heads, q_heads, dim, page, first):
    """Sizes on the side of the rules where a group's rows share tiles, of 16 and of 128 rows; beside the long group
    one that shares nothing, one with a shorter prefix, an empty sequence."""
    rng = np.random.default_rng(dim + q_heads)
    prefix, width, new = first
    groups = [(prefix, [(37 * i) % 150 for i in range(width)], [1 + i % new for i in range(width)]), (0, [300], [1]),
              (page * (600 // page) + 5, [0, 90, 3], [1, 0, new])]
    c = Answers(rng, groups, n_heads, dim, page)
    say(f"bl_attention_shared together {first} heads={n_heads}/{q_heads} dim={dim} page={page}")
    assert together(c, q_heads)
    q = heads(rng, c.total, q_heads, dim)
    check(c, q)
    c.table[:width, 3] = -1             # a hole in the prefix, and one sequence's own pages gone
    c.table[min(2, width - 1), prefix // page:] = -1
    c.va[c.table[0, 1]], c.ka[c.table[0, 2]] = 0, 0
    check(c, q)


@pytest.mark.parametrize("dim,page", [(64, 64), (128, 32)])
def test_long_rests_behind_a_prefix(dim, page):
    """Prefix and rests both with many rows and steps, on workgroups of two teams."""
    rng = np.random.default_rng(dim)
    c = Answers(rng, [(20000, [2100 + 7 * i for i in range(30)], [9 - i % 2 for i in range(30)])], 1, dim, page)
    say(f"bl_attention_shared long rests dim={dim}")
    assert together(c, 8)
    check(c, heads(rng, c.total, 8, dim))


def test_nan_in_a_prefix_taken_together():
    rng = np.random.default_rng(6)
    c = Answers(rng, [(9000, [i for i in range(30)], [1] * 30), (9000, [3, 70], [1, 1])], 2, 64, 64)
    q = heads(rng, c.total, 8, 64)
    assert together(c, 8)
    say("bl_attention_shared NaN, together")

    def attend():
        cache, batch = c.device()
        return bl.bl_attention_shared(cache, batch, c.shared(), bf16(_block.bits(q))).float().cpu().numpy()

    clean = attend()
    c.ka[c.table[0, 1], 1] = np.nan
    out = attend()
    assert np.isnan(out[:30, 4:]).all() and np.array_equal(out[30:], clean[30:]) and np.array_equal(out[:, :4], clean[:, :4])
    c.ka[c.table[0, 1], 1] = 1.0
    clean = attend()
    c.va[c.table[31, -1 if c.table[31, -1] >= 0 else 141], 0] = np.inf  # the last sequence's own last page
    q[3, 2, 5] = np.nan
    out = attend()
    assert np.isnan(out[31, :4]).all() and np.isnan(out[3, 2]).all()
    out[31, :4], out[3, 2] = clean[31, :4], clean[3, 2]
    assert np.array_equal(out, clean)


def test_captured_and_odd_integers_together():
    rng = np.random.default_rng(8)
    c = Answers(rng, [(9000, [5 * i for i in range(20)], [1] * 20), (640, [3, 70], [1, 1])], 2, 64, 64)
    q = bf16(_block.bits(heads(rng, c.total, 8, 64)))
    cache, batch = c.device()
    shared = c.shared()
    assert together(c, 8)
    say("bl_attention_shared captured, together")
    ws = torch.empty(bl.bl_attention_shared_workspace_bytes(cache, batch, shared, 8), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = bl.bl_attention_shared(cache, batch, shared, q, workspace=ws)
        graphs.append((g, out))
    prefix = shared.prefix.clone()
    for i in range(4):
        shared.prefix.copy_(prefix - 64 * i)  # the graph follows the device's integers
        expect = bl.bl_attention_shared(cache, batch, shared, q)
        ws.fill_(0xFF)
        graphs[i % 2][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[i % 2][1], expect)
    want = expect.float()
    for i, (group, far) in enumerate((([0, 99, -5], [1 << 30, -3]), ([-7, 2, 5], [128, 640]), ([20, 1, 5], [0, 9000]), ([0, 0, 0], [64, 64]),
                                      ([0, 20, 22], [9064, 1 << 30]))):
        odd = bl.KVShared(i32(group), i32(far), 20, 9000)
        need = bl.bl_attention_shared_workspace_bytes(cache, batch, odd, 8)
        walled, out, lse = Walled((need,), torch.uint8), Walled(tuple(q.shape), torch.bfloat16), Walled(tuple(q.shape[:2]), torch.float32)
        walled.t.zero_()
        bl.bl_attention_shared(cache, batch, odd, q, out=out.t, lse=lse.t, workspace=walled.t)
        torch.cuda.synchronize()
        assert walled.intact() and out.intact() and lse.intact()
    start = bl.KVBatch(batch.page_table, i32([-9, 1 << 30] + [5] * 20), batch.offsets, c.total, 1, batch.max_len)
    need = bl.bl_attention_shared_workspace_bytes(cache, start, shared, 8)
    walled, out = Walled((need,), torch.uint8), Walled(tuple(q.shape), torch.bfloat16)
    walled.t.zero_()
    bl.bl_attention_shared(cache, start, shared, q, out=out.t, workspace=walled.t)
    torch.cuda.synchronize()
    assert walled.intact() and out.intact() and torch.isfinite(want).all()


@pytest.mark.parametrize("width", [1, 5, 40])
def test_bounds_above_what_is_there(width):
    """max_prefix, max_group and max_len larger than any of the batch."""
    rng = np.random.default_rng(width)
    c = Answers(rng, [(200, [i for i in range(width)], [1] * width), (64, [3], [2])], 1, 64, 16)
    say(f"bl_attention_shared bounds width={width}")
    q = heads(rng, c.total, 4, 64)
    want = check(c, q)
    cache, batch = c.device()
    group, prefix = i32(np.concatenate([[0], np.cumsum(c.width)])), i32(c.prefix)
    stride = c.table.shape[1]
    wide = bl.KVBatch(batch.page_table, batch.start, batch.offsets, c.total, min(c.total, 9), stride * 16)
    out = bl.bl_attention_shared(cache, wide, bl.KVShared(group, prefix, width + 7, stride * 16), q=bf16(_block.bits(q)))
    # other splits, other sums: each within a bound of the exact value
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()


def test_missing_pages_and_rows_that_see_nothing():
    rng = np.random.default_rng(31)
    c = Answers(rng, [(128, [10, 40], [1, 2]), (64, [0, 3], [1, 1]), (80, [1, 2], [1, 1])], 2, 64, 16)
    for s in (0, 1):
        c.table[s, 2] = -1           # a hole in a prefix
    c.table[1, 9] = 1 << 30          # and behind it
    c.table[2:4, :] = -7             # a group with no page at all
    c.table[4:6, :4] = -1            # a prefix with none
    say("bl_attention_shared holes")
    check(c, heads(rng, c.total, 4, 64))


def test_nan_stays_with_those_that_see_it():
    rng = np.random.default_rng(5)
    c = Answers(rng, [(128, [10, 40], [1, 1]), (128, [3, 70], [1, 1])], 1, 64, 64)
    q = heads(rng, c.total, 2, 64)

    def attend():
        cache, batch = c.device()
        return bl.bl_attention_shared(cache, batch, c.shared(), bf16(_block.bits(q))).float().cpu().numpy()

    clean = attend()
    say("bl_attention_shared NaN")
    keep = c.ka.copy()
    c.ka[c.table[0, 1]] = np.nan                    # in the first prefix
    out = attend()
    assert np.isnan(out[:2]).all() and np.array_equal(out[2:], clean[2:])
    c.ka = keep.copy()
    c.ka[c.table[3, 2]] = np.inf                    # behind the second, one sequence's own
    out = attend()
    assert np.isnan(out[3]).all() and np.array_equal(out[:3], clean[:3])
    c.ka = keep
    q[1, 1, 7] = np.nan                             # a query
    out = attend()
    assert np.isnan(out[1, 1]).all()
    out[1, 1] = clean[1, 1]
    assert np.array_equal(out, clean)


def test_what_is_not_visible_does_not_matter():
    rng = np.random.default_rng(33)
    c = Answers(rng, [(96, [5, 20], [1, 1])], 1, 64, 16)
    q = heads(rng, c.total, 4, 64)
    say("bl_attention_shared unused data")
    a = check(c, q)
    used = set(c.table[0, :7]) | set(c.table[1, :8])
    for p in range(len(c.ka)):
        if p not in used:
            c.ka[p], c.va[p] = np.nan, np.inf
    assert torch.equal(check(c, q), a)


@pytest.mark.parametrize("width", [1, 30])
def test_sharp_and_flat_softmax_and_scales_far_apart(width):
    rng = np.random.default_rng(43)
    c = Answers(rng, [(500, list(range(width)), [1] * width)], 1, 64, 64)
    q = heads(rng, c.total, 4, 64)
    say("bl_attention_shared sharp and flat")
    check(c, q, scale=4.0)
    check(c, q, scale=0.0)
    check(c, q, scale=-0.125)
    c.va[:] = (np.float32(2) ** rng.integers(-40, 1, c.va.shape)).astype(np.float32)
    check(c, q)


def test_strided_queries_another_stream_and_a_graph():
    rng = np.random.default_rng(47)
    c = Answers(rng, [(256, [70, 3, 9], [1, 1, 2])], 2, 64, 16)
    qkv = heads(rng, c.total, 8, 64)
    qd = bf16(_block.bits(qkv))[:, 2:6]
    say("bl_attention_shared strided")
    want = check(c, qkv[:, 2:6], q_device=qd)
    cache, batch = c.device()
    shared = c.shared()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = bl.bl_attention_shared(cache, batch, shared, qd)
    side.synchronize()
    assert torch.equal(other, want)
    ws = torch.empty(bl.bl_attention_shared_workspace_bytes(cache, batch, shared, 4), dtype=torch.uint8, device=DEV)
    graphs = []
    for _ in range(2):  # over one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = bl.bl_attention_shared(cache, batch, shared, qd, workspace=ws)
        graphs.append((g, out))
    start = batch.start.clone()
    for i in range(4):
        batch.start.copy_(start - (i % 3))  # the graph follows the device's lengths
        expect = bl.bl_attention_shared(cache, batch, shared, qd)
        ws.fill_(0xFF)
        graphs[i % 2][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[i % 2][1], expect)


def test_device_integers_out_of_bounds_stay_inside_the_buffers():
    rng = np.random.default_rng(53)
    c = Answers(rng, [(128, [10, 40, 3], [1, 2, 1]), (64, [0, 3], [1, 1])], 2, 64, 16)
    cache, batch = c.device()
    q = bf16(_block.bits(heads(rng, c.total, 4, 64)))
    say("bl_attention_shared odd integers")
    for group, prefix, start in (([0, 99, -5], [1 << 30, -3], None), ([-7, 2, 5], [128, 640], None), ([3, 1, 5], [0, 64], None),
                                 ([0, 3, 5], [128, 64], [-9, 1 << 30, 0, 5, 64]), ([0, 0, 0], [64, 64], None)):
        shared = bl.KVShared(i32(group), i32(prefix), 3, 128)
        b = batch if start is None else bl.KVBatch(batch.page_table, i32(start), batch.offsets, c.total, 2, batch.max_len)
        need = bl.bl_attention_shared_workspace_bytes(cache, b, shared, 4)
        ws, out, lse = Walled((need,), torch.uint8), Walled(tuple(q.shape), torch.bfloat16), Walled(tuple(q.shape[:2]), torch.float32)
        ws.t.zero_()
        bl.bl_attention_shared(cache, b, shared, q, out=out.t, lse=lse.t, workspace=ws.t)
        torch.cuda.synchronize()
        assert ws.intact() and out.intact() and lse.intact()


def test_cache_past_two_to_the_32_bytes():
    """A prefix whose pages lie behind 4 GiB of keys."""
    say("bl_attention_shared past 2^32 bytes")
    pages, n_heads, page, dim = 9000, 4, 64, 256
    cache = bl.KVCache.empty(pages, n_heads, page, dim, DEV)  # 590 MB of each per 1000 pages
    g = torch.Generator(device=DEV).manual_seed(3)
    cache.k[-40:] = torch.randint(-127, 128, (40, n_heads, page, dim), generator=g, device=DEV, dtype=torch.int8)
    cache.v[-40:] = torch.randint(-127, 128, (40, n_heads, page, dim), generator=g, device=DEV, dtype=torch.int8)
    cache.k_absmax[-40:], cache.v_absmax[-40:] = 2.0, 3.0
    table = torch.tensor([[pages - 1 - i for i in range(16)] + [pages - 20, 0], [pages - 1 - i for i in range(16)] + [pages - 21, 0]],
                         dtype=torch.int32, device=DEV)
    q = torch.randn((2, 8, dim), generator=g, device=DEV).to(torch.bfloat16)
    batch = bl.KVBatch(table, i32([1050, 1024]), i32([0, 1, 2]), 2, 1, 1051)
    out = bl.bl_attention_shared(cache, batch, bl.KVShared(i32([0, 2]), i32([1024]), 2, 1024), q)
    want = bl.bl_attention(cache, batch, q)
    assert want.float().abs().max() > 0.01
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
