"""GPU checks of the attention at the ends of its number ranges, in both of its
kernels (one new token; 40 over more than 32 steps of keys), against the 64-bit
softmax with the bounds of _block.attention."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, host, say
from test_gpu_attention import check
from test_gpu_kv_cache import Case, heads

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

STEPS = [(200, 1), (1500, 1), (2200, 40)]


def zero_values(c, i):
    """Page i of the sequence holds zeros, as bl_kv_append writes them."""
    c.v[c.table[0, i]] = 0
    c.va[c.table[0, i]] = 0


@pytest.mark.parametrize("ctx,new", STEPS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("small", [-20, -40, -60])
def test_page_of_zero_values_among_small_ones(ctx, new, page, small):
    """Its weights count in the softmax's sum, and the others keep theirs."""
    rng = np.random.default_rng(ctx + page - small)
    c = Case(rng, [ctx], [new], 1, 64, page)
    c.va *= np.float32(2.0 ** small)
    zero_values(c, 0)
    zero_values(c, 2)
    say(f"bl_attention zero page among 2^{small}, ctx={ctx} new={new} page={page}")
    check(c, heads(rng, c.total, 2, 64))


@pytest.mark.parametrize("ctx,new", STEPS)
@pytest.mark.parametrize("page", [16, 64])
def test_page_of_zero_values_that_scores_far_above_the_rest(ctx, new, page):
    """Keys along the queries: scores some 50 bits above the others', whose small contributions are all there is."""
    rng = np.random.default_rng(ctx + page)
    c = Case(rng, [ctx], [new], 1, 64, page)
    one = heads(rng, 64)
    top = np.abs(one).max()
    p = c.table[0, 1]
    c.k[p] = np.rint(one * (127 / top)).astype(np.int8)
    c.ka[p] = 1.5 * top
    zero_values(c, 1)
    say(f"bl_attention zero page far above, ctx={ctx} new={new} page={page}")
    check(c, np.broadcast_to(one, (c.total, 2, 64)).copy())


@pytest.mark.parametrize("ctx,new", STEPS)
def test_codes_of_a_page_without_a_scale_stand_for_zeros(ctx, new):
    rng = np.random.default_rng(ctx)
    c = Case(rng, [ctx], [new], 1, 64, 16)
    c.va[c.table[0, 1]] = 0
    c.va[c.table[0, 5]] = np.float32(1e-42)  # no normal number
    say(f"bl_attention page without a scale, ctx={ctx} new={new}")
    check(c, heads(rng, c.total, 2, 64))


@pytest.mark.parametrize("ctx,new", STEPS)
def test_only_pages_of_zero_values(ctx, new):
    rng = np.random.default_rng(ctx + 1)
    c = Case(rng, [ctx], [new], 1, 64, 16)
    c.v[:], c.va[:] = 0, 0
    say(f"bl_attention only zero pages, ctx={ctx} new={new}")
    assert not check(c, heads(rng, c.total, 2, 64)).any()


@pytest.mark.parametrize("ctx,new", STEPS)
@pytest.mark.parametrize("scale", [-1.0, -1e12, -1e30, -1e35, 1e30])
def test_scores_far_below_zero(ctx, new, scale):
    """One page is there, its keys along the queries: the one that scores highest (with a negative scale the
    shortest) takes everything, the next being a tenth of the score away.  Its score is right to the query's
    2^-15 and a few fp32 roundings."""
    rng = np.random.default_rng(ctx)
    c = Case(rng, [ctx], [new], 1, 64, 16)
    one = heads(rng, 64)
    top, p = np.abs(one).max(), c.table[0, 0]
    c.k[p, 0] = np.rint(rng.permutation(np.arange(1, 17))[:, None] / 16 * one * (127 / top))
    c.ka[p] = top
    c.table[0, 1:] = -1
    if scale == -1.0:
        one = one * np.float32(2.0 ** 8)
    q = np.broadcast_to(one, (c.total, 2, 64)).copy()
    cache, batch = c.device()
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    say(f"bl_attention scores far below zero, ctx={ctx} new={new} scale={scale}")
    out = bf16_bits_to_f64(host(bl.bl_attention(cache, batch, bf16(_block.bits(q)), scale=scale, lse=lse)))
    score = scale * (c.k[p, 0].astype(np.float64) @ one) * float(c.ka[p, 0]) / 127
    best = int(score.argmax())
    want = c.v[p, 0, best].astype(np.float64) * float(c.va[p, 0]) / 127
    assert (np.abs(out - want) <= np.abs(want) * (_block.U16 + 2.0 ** -10)).all()
    assert (np.abs(host(lse) / score[best] - 1) <= 2.0 ** -12).all()
