"""GPU checks of the attention's kernel for many rows (workgroups of 128 rows)
against the 64-bit softmax, with the bounds of _block.attention.

The sizes reach each of its forms: 64 rows and more over more than 32 steps of
64 keys (or enough work in shorter ones), one and two teams of waves, one and
several workgroups along the keys, heads up to 64, 128 and 256 elements, pages
of every size, windows, holes."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, host, say
from test_gpu_attention import check
from test_gpu_kv_cache import Case, heads, i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


def run(rng, ctx, new, n_heads, q_heads, dim, page, **kw):
    c = Case(rng, ctx, new, n_heads, dim, page)
    say(f"bl_attention prompts ctx={ctx} new={new} heads={n_heads}/{q_heads} dim={dim} page={page} {kw}")
    return check(c, heads(rng, c.total, q_heads, dim), **kw)


@pytest.mark.parametrize("ctx,new,n_heads,q_heads,dim,page", [
    ([2100], [40], 1, 2, 16, 64), ([2100, 30], [40, 64], 1, 2, 48, 16), ([2080], [33], 2, 8, 128, 32),
    ([2100], [64], 1, 1, 256, 64), ([2500, 0], [20, 3], 1, 4, 144, 128), ([2047], [130], 1, 3, 64, 256),
    ([2100], [77], 1, 1, 80, 16), ([0], [2200], 1, 1, 32, 32), ([2300, 2200, 2100], [70, 0, 1], 1, 2, 96, 64)])
def test_many_rows_over_many_keys(ctx, new, n_heads, q_heads, dim, page):
    run(np.random.default_rng(sum(ctx) + dim), ctx, new, n_heads, q_heads, dim, page)


def test_tiles_for_every_cu():
    """512 tiles of 128 rows: one team, no split; then 256: two teams, no split; the second sequences are short."""
    rng = np.random.default_rng(7)
    run(rng, [2050, 60, 1000, 2050, 2000, 5, 2050, 2050], [128] * 8, 8, 64, 16, 64)
    run(rng, [2050, 60, 1000, 2050], [128] * 4, 8, 64, 32, 64)


@pytest.mark.parametrize("window,sinks", [(2100, 0), (2100, 70), (2500, 4)])
def test_long_windows(window, sinks):
    run(np.random.default_rng(window + sinks), [4000, 2300], [60, 70], 1, 2, 64, 64, window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks,page", [(300, 0, 64), (250, 5, 16)])
def test_short_windows_over_enough_rows(window, sinks, page):
    """1000 tokens of 2 x 16 heads of 144: over the work at which 16-row workgroups hand over."""
    run(np.random.default_rng(window), [100], [1000], 16, 32, 144, page, window=window, sinks=sinks)


def test_holes_zero_pages_and_empty_rows():
    rng = np.random.default_rng(11)
    c = Case(rng, [2200, 2200, 2200], [40, 40, 40], 1, 64, 32)
    c.table[0, 3], c.table[0, 60], c.table[1, :] = -1, 1 << 30, -7  # holes; a sequence with no page at all
    c.table[0, 68:] = -1                                            # and none where the new tokens are
    for i in range(20):
        p = c.table[2, i]
        c.ka[p] = c.va[p] = 0
        c.k[p] = c.v[p] = 0
    say("bl_attention prompts with holes")
    check(c, heads(rng, c.total, 2, 64))
    check(c, heads(rng, c.total, 2, 64), window=2100, sinks=40)


def test_first_keys_missing_then_seen():
    """Rows that see nothing in their first steps start late, at scores far from zero."""
    rng = np.random.default_rng(12)
    c = Case(rng, [2200], [40], 1, 64, 16)
    c.table[0, :100] = -1
    q = heads(rng, c.total, 2, 64)
    say("bl_attention prompts, late start")
    check(c, q, scale=3.0)
    check(c, q, scale=-3.0)


def test_unused_data_does_not_matter():
    rng = np.random.default_rng(13)
    c = Case(rng, [2105], [35], 1, 64, 16)
    used, q = set(c.table[0]), heads(rng, c.total, 4, 64)
    a = check(c, q)
    for p in range(len(c.ka)):
        if p not in used:
            c.ka[p], c.va[p] = np.nan, np.inf
    end = 2105 + 35
    c.k[c.table[0, (end - 1) // 16], :, (end - 1) % 16 + 1:] = 127
    c.v[c.table[0, (end - 1) // 16], :, (end - 1) % 16 + 1:] = -128
    assert torch.equal(check(c, q), a)


def test_scales_far_apart_sharp_and_flat():
    rng = np.random.default_rng(14)
    c = Case(rng, [2200], [40], 1, 64, 16)
    c.va[:] = (np.float32(2) ** rng.integers(-40, 1, c.va.shape)).astype(np.float32)
    c.va[c.table[0, 30]] = np.float32(2.0 ** 30)
    q = heads(rng, c.total, 2, 64)
    say("bl_attention prompts, scales")
    check(c, q)
    c.va[:] = 1
    check(c, q, scale=4.0)
    check(c, q, scale=0.0)
    check(c, np.zeros_like(q))


def test_workspace_covers_every_window():
    """A window can need more workgroups along the keys than its lack: the
    workspace that the call asks for holds them all."""
    rng = np.random.default_rng(15)
    for ctx, new, q_heads, window in [(4480, 33, 2, 4352), (6000, 64, 1, 2176), (4000, 1, 4, 1100), (9000, 20, 4, 4000)]:
        run(rng, [ctx], [new], 1, q_heads, 16, 64, window=window)


@pytest.mark.parametrize("tokens", [512, 513, 1024, 1025])
@pytest.mark.parametrize("dim,seqs", [(256, 1), (192, 2), (128, 1), (64, 3)])
def test_either_side_of_a_split_along_the_keys(tokens, dim, seqs):
    """8 and 9 (long heads), 16 and 17 steps: one workgroup and several; the other sequences are short."""
    run(np.random.default_rng(tokens + dim), [tokens - 1] + [30] * (seqs - 1), [1] * seqs, 2, 8, dim, 64)


@pytest.mark.parametrize("new", [97, 100, 103])
def test_either_side_of_the_kernel_for_many_rows(new):
    """12 heads of 128 over 10 and 11 steps: 23040 to 27456 tile steps of 16 rows."""
    run(np.random.default_rng(new), [540, 540, 440, 540], [new, new, 3, new], 12, 48, 128, 32)


def test_prompts_past_32_bits():
    """The same sequence in the first pages of a cache and past its 2^32-th byte gives the same bits."""
    rng = np.random.default_rng(16)
    n_heads, page, dim, ctx, new = 8, 64, 128, 2050, 64
    need = -(-(ctx + new) // page)
    pages = (1 << 32) // (n_heads * page * dim) + 2 * need
    c = Case(rng, [ctx], [new], n_heads, dim, page, spare=0)
    c.table = np.arange(need)[None]
    say("bl_attention prompts past 2^32 bytes")
    big = [torch.empty((pages, n_heads, page, dim), dtype=torch.int8, device=DEV) for _ in range(2)]
    top = [torch.ones((pages, n_heads), device=DEV) for _ in range(2)]
    table = np.stack([np.arange(need), pages - 1 - np.arange(need)])
    for t, a, codes, absmax in zip(big, top, (c.k, c.v), (c.ka, c.va)):
        for row in table:
            t[torch.from_numpy(row).to(DEV)] = torch.from_numpy(codes).to(DEV)
            a[torch.from_numpy(row).to(DEV)] = torch.from_numpy(absmax).to(DEV)
    batch = bl.KVBatch(i32(table), i32([ctx, ctx]), i32([0, new, 2 * new]), 2 * new, new, ctx + new)
    q = heads(rng, new, 32, dim)
    one = bf16(_block.bits(q))
    out = bl.bl_attention(bl.KVCache(*big, *top), batch, torch.cat([one, one]))
    torch.cuda.synchronize()
    assert torch.equal(out[:new], out[new:])
    want, _, bound, _ = _block.attention(q, c.k, c.ka, c.v, c.va, c.table, c.start, c.offsets,
                                         np.float64(np.float32(dim ** -0.5)))
    assert (np.abs(bf16_bits_to_f64(host(out[:new])) - want) <= bound + _block.U16 * (np.abs(want) + bound)).all()
