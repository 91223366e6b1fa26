"""GPU checks of the attention's kernel for many rows (workgroups of 128 rows)
against the 64-bit softmax, with the bounds of _block.attention.

The sizes reach each of its forms: 64 rows and more over more than 32 steps of
64 keys (or enough work in shorter ones), one and two teams of waves, one and
several workgroups along the keys, heads up to 64, 128 and 256 elements, pages
of every size, windows, holes."""
import numpy as np
import pytest
import torch

from _gpu import say
from test_gpu_attention import check
from test_gpu_kv_cache import Case, heads

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
