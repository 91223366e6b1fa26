"""GPU checks of the attention over the 8-bit cache against a 64-bit softmax
over the same codes; bounds as derived in _block.attention, plus bf16's unit
for the output's rounding."""
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


def check(c, q, scale=None, window=0, sinks=0, q_device=None):
    cache, batch = c.device()
    dim = c.k.shape[3]
    scale = dim ** -0.5 if scale is None else scale
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    qd = bf16(_block.bits(q)) if q_device is None else q_device
    out = bl.bl_attention(cache, batch, qd, scale=scale, window=window, sinks=sinks, lse=lse,
                          out=torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV))
    want, want_lse, bound, lse_bound = _block.attention(q, c.k, c.ka, c.v, c.va, c.table, c.start, c.offsets,
                                                        np.float64(np.float32(scale)), window, sinks)
    got, got_lse = bf16_bits_to_f64(host(out)), host(lse).astype(np.float64)
    off = np.abs(got - want) - (bound + _block.U16 * (np.abs(want) + bound))
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} outputs outside their bound, by up to {off.max():.3g}"
    none = np.isinf(want_lse)
    assert (got[none] == 0).all() and (got_lse[none] == -np.inf).all()
    assert (np.abs(got_lse[~none] - want_lse[~none]) <= lse_bound[~none]).all()
    again = bl.bl_attention(cache, batch, qd, scale=scale, window=window, sinks=sinks)
    assert torch.equal(again, out)
    return out


GEOMETRY = [  # heads, q heads, dim, page
    (2, 2, 64, 16), (1, 4, 128, 64), (2, 10, 128, 32), (1, 3, 80, 64), (3, 3, 16, 128), (1, 8, 48, 16), (1, 20, 64, 64),
    (2, 4, 256, 64), (1, 2, 144, 32), (1, 1, 192, 256)]


@pytest.mark.parametrize("n_heads,q_heads,dim,page", GEOMETRY)
@pytest.mark.parametrize("ctx,new", [([0], [1]), ([62, 63, 64, 15], [1, 1, 1, 1]), ([300, 5, 0], [1, 2, 1]), ([40, 0, 7], [3, 0, 20]),
                                     ([0, 130], [70, 5])])
def test_attention_matches_reference(n_heads, q_heads, dim, page, ctx, new):
    rng = np.random.default_rng(sum(ctx) * 3 + sum(new) + dim + q_heads)
    c = Case(rng, ctx, new, n_heads, dim, page)
    say(f"bl_attention ctx={ctx} new={new} heads={n_heads}/{q_heads} dim={dim} page={page}")
    check(c, heads(rng, c.total, q_heads, dim))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 4), (100, 70), (1000, 0), (65, 16), (1 << 40, 0)])
@pytest.mark.parametrize("ctx,new", [([0], [1]), ([500, 90], [1, 1]), ([200, 0], [50, 90])])
def test_window_and_sinks(window, sinks, ctx, new):
    rng = np.random.default_rng(window % 1000 + sinks + sum(ctx))
    c = Case(rng, ctx, new, 2, 64, 32)
    say(f"bl_attention window={window} sinks={sinks} ctx={ctx} new={new}")
    check(c, heads(rng, c.total, 6, 64), window=window, sinks=sinks)


@pytest.mark.parametrize("ctx,new,dim", [([20000], [1], 128), ([9000, 30000, 3, 700], [1, 1, 1, 1], 64), ([5000], [6], 256),
                                         ([2500], [300], 128)])
def test_long_sequences(ctx, new, dim):
    """Many workgroups along the keys, joined afterwards."""
    rng = np.random.default_rng(sum(ctx))
    c = Case(rng, ctx, new, 1, dim, 64)
    say(f"bl_attention long ctx={ctx} new={new} dim={dim}")
    check(c, heads(rng, c.total, 4, dim))


@pytest.mark.parametrize("new", [1, 40])
def test_missing_pages_are_skipped_and_empty_rows_give_zeros(new):
    rng = np.random.default_rng(31 + new)
    c = Case(rng, [100, 60, 10], [new, new, new], 2, 64, 16)
    c.table[0, 2], c.table[0, 5], c.table[1, :] = -1, 1 << 30, -7  # holes; a sequence with no page at all
    c.ka[c.table[2, 0]] = 0  # a page of zeros
    c.va[c.table[2, 0]] = 0
    c.k[c.table[2, 0]] = 0
    c.v[c.table[2, 0]] = 0
    say(f"bl_attention holes new={new}")
    check(c, heads(rng, c.total, 4, 64))


@pytest.mark.parametrize("new", [1, 33])
def test_what_is_not_visible_does_not_matter(new):
    """Unused pages and the rest of the last page hold anything, NaN scales included."""
    rng = np.random.default_rng(33)
    c = Case(rng, [37], [new], 1, 64, 16)
    used = set(c.table[0])
    q = heads(rng, c.total, 4, 64)
    say("bl_attention unused data")
    a = check(c, q)
    for p in range(len(c.ka)):
        if p not in used:
            c.ka[p], c.va[p] = np.nan, np.inf
    last = c.table[0, (37 + new - 1) // 16]
    c.k[last, :, (37 + new - 1) % 16 + 1:] = 127
    c.v[last, :, (37 + new - 1) % 16 + 1:] = -128
    assert torch.equal(check(c, q), a)


@pytest.mark.parametrize("new", [1, 20])
def test_scales_far_apart(new):
    """Pages whose values differ by 2^40 in scale: neither side is lost."""
    rng = np.random.default_rng(41)
    c = Case(rng, [200], [new], 1, 64, 16)
    c.va[:] = (np.float32(2) ** rng.integers(-40, 1, c.va.shape)).astype(np.float32)
    c.va[c.table[0, 3]] = np.float32(2.0 ** 30)
    say("bl_attention scales far apart")
    check(c, heads(rng, c.total, 2, 64))
    c.va[:] = np.float32(2.0 ** -60)
    check(c, heads(rng, c.total, 2, 64))


@pytest.mark.parametrize("new", [1, 20])
def test_sharp_and_flat_softmax(new):
    rng = np.random.default_rng(43)
    c = Case(rng, [500], [new], 1, 64, 64)
    q = heads(rng, c.total, 4, 64)
    say("bl_attention sharp and flat")
    check(c, q, scale=4.0)       # one key takes nearly all
    check(c, q, scale=0.0)       # every key alike
    check(c, q, scale=-0.125)
    check(c, np.zeros_like(q))
    check(c, _block.bf16_round(q * np.float32(2.0 ** -90)))


def test_strided_queries_and_another_stream():
    rng = np.random.default_rng(47)
    c = Case(rng, [70, 3], [1, 5], 2, 64, 16)
    qkv = heads(rng, c.total, 8, 64)
    qd = bf16(_block.bits(qkv))[:, 2:6]
    say("bl_attention strided")
    out = check(c, qkv[:, 2:6], q_device=qd)
    cache, batch = c.device()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = bl.bl_attention(cache, batch, qd)
    side.synchronize()
    assert torch.equal(other, out)


def test_captured_decode_step():
    """Append and attention of one token in a graph: every replay sees the
    positions that stand in device memory at that time."""
    rng = np.random.default_rng(53)
    steps, ctx = 5, 4100
    c = Case(rng, [ctx], [steps], 1, 64, 64)
    cache, _ = c.device()
    eager_cache, _ = Case.device(c)[0], None
    cache = bl.KVCache(eager_cache.k.clone(), eager_cache.v.clone(), eager_cache.k_absmax.clone(), eager_cache.v_absmax.clone())
    qkv = bf16(_block.bits(heads(rng, steps, 6, 64)))
    rope = bl.Rope(bl.bl_rope_frequencies(64).to(DEV))
    start, offsets = i32([ctx]), i32([0, 1])
    batch = bl.KVBatch(i32(c.table), start, offsets, 1, 1, ctx + steps)
    one = qkv[:1].clone()
    q_out, out = torch.empty((1, 4, 64), dtype=torch.bfloat16, device=DEV), torch.empty((1, 4, 64), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(bl.bl_attention_workspace_bytes(cache, batch, 4), 16), dtype=torch.uint8, device=DEV)
    say("bl_kv_append + bl_attention captured")

    def step(kv):
        bl.bl_kv_append(kv, batch, one[:, 4:5], one[:, 5:6], rope=rope, q=one[:, :4], q_out=q_out)
        bl.bl_attention(kv, batch, q_out, out=out, workspace=ws)

    want = []
    for i in range(steps):
        one.copy_(qkv[i:i + 1])
        start.fill_(ctx + i)
        step(eager_cache)
        want.append(out.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    one.copy_(qkv[:1])
    start.fill_(ctx)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(cache)
    for i in range(steps):
        one.copy_(qkv[i:i + 1])
        start.fill_(ctx + i)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), f"replay {i}"
    assert torch.equal(cache.k, eager_cache.k) and torch.equal(cache.v_absmax, eager_cache.v_absmax)


def test_cache_longer_than_32_bits():
    """Pages past 2^32 bytes of the cache are found: the same sequence in the
    first pages and in the last ones gives the same bits."""
    rng = np.random.default_rng(59)
    n_heads, page, dim = 8, 64, 128
    pages = (1 << 32) // (n_heads * page * dim) + 40
    c = Case(rng, [300, 300], [1, 1], n_heads, dim, page, spare=0)
    say("bl_attention, bl_kv_append and bl_kv_read past 2^32 bytes")
    big = [torch.empty((pages, n_heads, page, dim), dtype=torch.int8, device=DEV) for _ in range(2)]
    top = [torch.ones((pages, n_heads), device=DEV) for _ in range(2)]
    table = np.stack([np.arange(5), pages - 1 - np.arange(5)])
    for t, a, codes, absmax in zip(big, top, (c.k, c.v), (c.ka, c.va)):
        for row in table:
            t[torch.from_numpy(row).to(DEV)] = torch.from_numpy(codes[:5]).to(DEV)
            a[torch.from_numpy(row).to(DEV)] = torch.from_numpy(absmax[:5]).to(DEV)
    cache = bl.KVCache(*big, *top)
    batch = bl.KVBatch(i32(table), i32([300, 300]), i32([0, 1, 2]), 2, 1, 301)
    one = bf16(_block.bits(np.repeat(heads(rng, 1, 32, dim), 2, axis=0)))
    kv = one[:, :n_heads].contiguous()
    bl.bl_kv_append(cache, batch, kv, kv)
    rk, rv = bl.bl_kv_read(cache, batch)
    out = bl.bl_attention(cache, batch, one)
    torch.cuda.synchronize()
    assert torch.equal(rk[0], rk[1]) and torch.equal(rv[0], rv[1]) and torch.equal(out[0], out[1])
    assert (rk[0].float() - kv[0].float()).abs().max() <= kv.float().abs().max().clamp(min=4.0) / 127
    c.table, c.k, c.ka, c.v, c.va = table[:1], *(host(t[:5]) for t in (cache.k, cache.k_absmax, cache.v, cache.v_absmax))
    c.start, c.offsets = np.array([300]), np.array([0, 1])
    want, _, bound, _ = _block.attention(bf16_bits_to_f64(host(one[:1])), c.k, c.ka, c.v, c.va, c.table, c.start, c.offsets,
                                         np.float64(np.float32(dim ** -0.5)))
    assert (np.abs(bf16_bits_to_f64(host(out[:1])) - want) <= bound + _block.U16 * (np.abs(want) + bound)).all()


def test_workspace_on_the_host_is_refused():
    c = Case(np.random.default_rng(61), [40], [1], 2, 64, 16)
    cache, batch = c.device()
    q = bf16(_block.bits(heads(c.rng, 1, 4, 64)))
    with pytest.raises(ValueError, match="workspace"):
        bl.bl_attention(cache, batch, q, workspace=torch.empty(1 << 16, dtype=torch.uint8))
