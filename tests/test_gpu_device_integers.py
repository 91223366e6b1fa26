"""Positions and offsets on the device that break the bounds the host was
given: no access leaves a buffer (bytes around each are checked), and what is
inside the bounds is still right.  Attention sees no position from max_len on,
which is what a page table that ends there gives."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, host, say
from test_gpu_kv_cache import Case, heads, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

ROUND = 4096  # bytes before and after each buffer


class Walled:
    """A tensor in the middle of a buffer whose other bytes stay as they are."""

    def __init__(self, shape, dtype, like=None):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.all = torch.full((n + 2 * ROUND,), 0xA5, dtype=torch.uint8, device=DEV)
        self.n = n
        self.t = self.all[ROUND:ROUND + n].view(dtype).view(shape)
        if like is not None:
            self.t.copy_(like)

    def intact(self):
        return bool((self.all[:ROUND] == 0xA5).all()) and bool((self.all[ROUND + self.n:] == 0xA5).all())


def attend(c, q, start, offsets, max_new, max_len, window=0, sinks=0):
    cache, _ = c.device()
    tokens = q.shape[0]
    batch = bl.KVBatch(i32(c.table), i32(start), i32(offsets), tokens, max_new, max_len)
    need = bl.bl_attention_workspace_bytes(cache, batch, q.shape[1])
    ws, out, lse = Walled((need,), torch.uint8), Walled(q.shape, torch.bfloat16), Walled(q.shape[:2], torch.float32)
    out.t.fill_(9.0)
    lse.t.fill_(9.0)
    torch.cuda.synchronize()
    bl.bl_attention(cache, batch, bf16(_block.bits(q)), window=window, sinks=sinks, out=out.t, lse=lse.t, workspace=ws.t)
    torch.cuda.synchronize()
    assert ws.intact() and out.intact() and lse.intact()
    return bf16_bits_to_f64(host(out.t)), host(lse.t).astype(np.float64)


def compare(c, q, got, lse, start, offsets, max_len, window, sinks):
    """Against the 64-bit softmax over a table that ends at max_len (a whole number of pages)."""
    table = np.where(np.arange(c.table.shape[1]) < max_len // c.page, c.table, -1)
    table = np.concatenate([table, np.full((len(start), 4096), -1)], axis=1)
    want, want_lse, bound, lse_bound = _block.attention(q, c.k, c.ka, c.v, c.va, table, start, offsets,
                                                        np.float64(np.float32(q.shape[2] ** -0.5)), window, sinks)
    assert (np.abs(got - want) <= bound + _block.U16 * (np.abs(want) + bound)).all()
    none = np.isinf(want_lse)
    assert (got[none] == 0).all() and (lse[none] == -np.inf).all()
    assert (np.abs(lse[~none] - want_lse[~none]) <= lse_bound[~none]).all()


@pytest.mark.parametrize("start,new,max_len,window,sinks", [
    ([200, 90], [1, 1], 96, 0, 0),          # one workgroup per tile, no workspace
    ([1500, 30], [2, 2], 992, 0, 0),        # the same, a step from the split
    ([5000, 2000], [1, 1], 3072, 0, 0),     # several workgroups along the keys
    ([5000, 300], [70, 70], 3072, 0, 0),    # workgroups of 128 rows
    ([1040, 1000], [40, 40], 1024, 0, 0),   # positions on either side of max_len
    ([3060, 3000], [70, 20], 3072, 0, 0),
    ([5000, 100], [1, 1], 3072, 64, 0),     # the window lies past max_len: nothing is seen
    ([5000, 100], [70, 70], 3072, 2400, 5),  # only the first tokens
    ([3100, 3000], [3, 3], 3072, 100, 40),
])
@pytest.mark.parametrize("page", [16, 64])
def test_attention_past_max_len(start, new, max_len, window, sinks, page):
    if max_len % page:
        max_len -= max_len % page
    rng = np.random.default_rng(sum(start) + new[0] + window)
    c = Case(rng, [5200, 5200], [1, 1], 2, 64, page)  # the table has room for all of these positions
    q = heads(rng, sum(new), 4, 64)
    offsets = np.array([0, new[0], sum(new)])
    say(f"bl_attention start={start} new={new} max_len={max_len} window={window} sinks={sinks} page={page}")
    got, lse = attend(c, q, start, offsets, max(new), max_len, window, sinks)
    compare(c, q, got, lse, start, offsets, max_len, window, sinks)


@pytest.mark.parametrize("new", [1, 70])
def test_attention_of_positions_far_outside(new):
    rng = np.random.default_rng(new)
    c = Case(rng, [2500, 2500], [new, new], 1, 64, 64)
    q = heads(rng, 2 * new, 2, 64)
    offsets = np.array([0, new, 2 * new])
    say(f"bl_attention far outside new={new}")
    got, lse = attend(c, q, [-(1 << 31), (1 << 31) - 1], offsets, new, 2560)
    # a negative start is 0; the second sequence sees all of 0 .. max_len - 1
    compare(c, q, got, lse, [0, 1 << 16], offsets, 2560, 0, 0)


@pytest.mark.parametrize("offsets,same", [([0, 6, 3, 9], [(0, 0, 3)]), ([-5, 3, 1 << 30, 1 << 30], [(0, 0, 3), (1, 3, 9)]),
                                          ([4, 2, -1, -(1 << 31)], [])])
def test_attention_with_offsets_out_of_order(offsets, same):
    """`same`: (sequence, first, last) rows that one sequence alone writes."""
    rng = np.random.default_rng(3)
    c = Case(rng, [100, 60, 30], [6, 6, 6], 2, 64, 16)
    q = heads(rng, 9, 4, 64)
    say(f"bl_attention offsets={offsets}")
    got, lse = attend(c, q, c.start, offsets, 6, 106)
    for s, first, last in same:
        own = Case(rng, [int(c.start[s])], [last - first], 2, 64, 16)
        own.table, own.k, own.v, own.ka, own.va = c.table[s:s + 1], c.k, c.v, c.ka, c.va
        compare(own, q[first:last], got[first:last], lse[first:last], own.start, np.array([0, last - first]), 112, 0, 0)


@pytest.mark.parametrize("start,offsets", [([-9, 1 << 30], [0, 20, 40]), ([90, 95], [0, 20, 40]), ([3, 5], [0, 50, 7]),
                                           ([(1 << 31) - 1, 0], [-3, 1 << 30, 4])])
def test_cache_calls_with_integers_out_of_range(start, offsets):
    """A table of 96 positions: what lies past it is neither written nor read."""
    rng = np.random.default_rng(7)
    c = Case(rng, [80, 80], [16, 16], 2, 64, 16)
    k, v, ka, va = (Walled(a.shape, t, torch.from_numpy(a)) for a, t in (
        (c.k, torch.int8), (c.v, torch.int8), (c.ka, torch.float32), (c.va, torch.float32)))
    cache = bl.KVCache(k.t, v.t, ka.t, va.t)
    batch = bl.KVBatch(i32(c.table), i32(start), i32(offsets), 40, 20, 96)
    x, q = heads(rng, 40, 4, 64), heads(rng, 40, 6, 64)
    q_out, rk, rv = (Walled(s, torch.bfloat16) for s in ((40, 6, 64), (40, 2, 64), (40, 2, 64)))
    say(f"bl_kv_append, bl_kv_read start={start} offsets={offsets}")
    torch.cuda.synchronize()
    rope = bl.Rope(bl.bl_rope_frequencies(64).to(DEV))
    xd = bf16(_block.bits(x))
    bl.bl_kv_append(cache, batch, xd[:, :2], xd[:, 2:], rope=rope, q=bf16(_block.bits(q)), q_out=q_out.t)
    bl.bl_kv_read(cache, batch, k=rk.t, v=rv.t)
    torch.cuda.synchronize()
    assert all(w.intact() for w in (k, v, ka, va, q_out, rk, rv))
    untouched = [p for p in range(len(c.ka)) if p not in set(c.table.ravel())]
    np.testing.assert_array_equal(host(v.t)[untouched], c.v[untouched])
    if list(offsets) == [0, 20, 40]:  # each row has one writer: the values are those of the rows inside the table
        first = [max(0, a) for a in start]
        inside = [max(0, min(20, 96 - a)) for a in first]
        rows = np.concatenate([x[0:inside[0], 2:], x[20:20 + inside[1], 2:]])
        at = np.array([0, inside[0], sum(inside)])
        want_v, want_va = _block.append(c.v, c.va, c.table, first, at, rows)
        np.testing.assert_array_equal(host(v.t), want_v)
        np.testing.assert_array_equal(host(va.t), want_va)
        back = _block.read(want_v, want_va, c.table, first, at)
        got = host(rv.t)
        np.testing.assert_array_equal(got[0:inside[0]], _block.bits(back[:inside[0]]))
        np.testing.assert_array_equal(got[20:20 + inside[1]], _block.bits(back[inside[0]:]))
        assert (got[inside[0]:20] & 0x7FFF == 0).all() and (got[20 + inside[1]:] & 0x7FFF == 0).all()


def test_captured_step_replayed_past_its_table():
    """A graph that moves its own positions, replayed past max_len: the same as eager calls at those positions, the
    bytes around the cache and the workspace as they were."""
    rng = np.random.default_rng(17)
    c = Case(rng, [1010, 500], [1, 1], 2, 64, 16)
    assert c.table.shape[1] * 16 == 1024  # the positions of the table; the second sequence's pages end at 512

    def fresh():
        k, v, ka, va = (Walled(a.shape, t, torch.from_numpy(a)) for a, t in (
            (c.k, torch.int8), (c.v, torch.int8), (c.ka, torch.float32), (c.va, torch.float32)))
        start = i32([1010, 500])
        batch = bl.KVBatch(i32(c.table), start, i32([0, 1, 2]), 2, 1, 1024)
        cache = bl.KVCache(k.t, v.t, ka.t, va.t)
        ws = Walled((max(16, bl.bl_attention_workspace_bytes(cache, batch, 4)),), torch.uint8)
        out, q_out = (torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        return cache, batch, start, (k, v, ka, va, ws), out, q_out

    qkv = bf16(_block.bits(heads(rng, 2, 8, 64)))
    rope = bl.Rope(bl.bl_rope_frequencies(64).to(DEV))

    def step(cache, batch, start, walls, out, q_out):
        bl.bl_kv_append(cache, batch, qkv[:, 4:6], qkv[:, 6:], rope=rope, q=qkv[:, :4], q_out=q_out)
        bl.bl_attention(cache, batch, q_out, out=out, workspace=walls[4].t)
        start.add_(1)

    say("captured step replayed past its table")
    eager, captured = fresh(), fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*captured)
    for i in range(20):  # positions 1010 .. 1029: the last six are past the table
        step(*eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[4], eager[4]) and torch.isfinite(captured[4].float()).all(), f"replay {i}"
    for a, b in zip(captured[3][:4], eager[3][:4]):
        assert a.intact() and b.intact() and torch.equal(a.t, b.t)
    assert captured[3][4].intact() and eager[3][4].intact()
