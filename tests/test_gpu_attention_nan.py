"""NaN and infinities in the attention's queries and page scales: they reach what
depends on them and nothing else."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, host, say
from test_gpu_kv_cache import Case, heads

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

STEPS = [([200, 90], [1, 1]), ([1500, 20], [1, 1]), ([2200, 2100], [40, 40])]  # the last: workgroups of 128 rows


def attend(c, q, **kw):
    cache, batch = c.device()
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    out = bl.bl_attention(cache, batch, bf16(_block.bits(q)), lse=lse, **kw)
    return out.float().cpu().numpy(), host(lse)


@pytest.mark.parametrize("ctx,new", STEPS)
@pytest.mark.parametrize("dim,element", [(64, 3), (64, 60), (128, 100), (256, 17)])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_query_that_is_not_finite(ctx, new, dim, element, value):
    rng = np.random.default_rng(dim + element)
    c = Case(rng, ctx, new, 1, dim, 64)
    q = heads(rng, c.total, 2, dim)
    clean, clean_lse = attend(c, q)
    row = (new[0] - 1, 1)
    q[row + (element,)] = value
    say(f"bl_attention query with {value} ctx={ctx} new={new} dim={dim}")
    out, lse = attend(c, q)
    assert np.isnan(out[row]).all() and np.isnan(lse[row])
    out[row], lse[row] = clean[row], clean_lse[row]
    np.testing.assert_array_equal(out, clean)
    np.testing.assert_array_equal(lse, clean_lse)


@pytest.mark.parametrize("ctx,new", STEPS)
@pytest.mark.parametrize("which", ["ka", "va"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("page", [16, 64])
def test_page_whose_scale_is_not_finite(ctx, new, which, value, page):
    rng = np.random.default_rng(page)
    c = Case(rng, ctx, new, 2, 64, page)
    q = heads(rng, c.total, 4, 64)
    clean, clean_lse = attend(c, q)
    getattr(c, which)[c.table[0, 1], 1] = value  # the first sequence's second page, second head
    say(f"bl_attention page with {which}={value} ctx={ctx} new={new} page={page}")
    out, lse = attend(c, q)
    rows = slice(0, new[0])
    assert np.isnan(out[rows, 2:]).all() and np.isnan(lse[rows, 2:]).all()
    out[rows, 2:], lse[rows, 2:] = clean[rows, 2:], clean_lse[rows, 2:]
    np.testing.assert_array_equal(out, clean)
    np.testing.assert_array_equal(lse, clean_lse)


@pytest.mark.parametrize("ctx,new,window", [([200], [1], 30), ([2230], [40], 2150)])
@pytest.mark.parametrize("which", ["ka", "va"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_page_outside_the_window_whose_scale_is_not_finite(ctx, new, window, which, value):
    """A page of 16 tokens that shares its step of 64 keys with visible ones."""
    rng = np.random.default_rng(5)
    c = Case(rng, ctx, new, 1, 64, 16)
    q = heads(rng, c.total, 2, 64)
    clean, clean_lse = attend(c, q, window=window)
    first = ctx[0] - window + 1
    page = first // 16 - 1
    assert page >= first // 64 * 4
    getattr(c, which)[c.table[0, page]] = value
    say(f"bl_attention masked page with {which}={value} ctx={ctx} new={new}")
    out, lse = attend(c, q, window=window)
    np.testing.assert_array_equal(out, clean)
    np.testing.assert_array_equal(lse, clean_lse)
