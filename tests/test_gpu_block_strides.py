"""Views whose axes of one element carry any stride: taken by every call that
takes heads, with the results of their dense copies."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import bf16, say
from test_gpu_kv_cache import Case, heads, i32, table

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


def odd(t, axes):
    """The same values in a view whose `axes` (of one element) have stride 3."""
    strides = [3 if a in axes else s for a, s in enumerate(t.stride())]
    return t.as_strided(t.shape, strides)


@pytest.mark.parametrize("tokens,n_heads,axes", [(1, 4, (0,)), (5, 1, (1,)), (1, 1, (0, 1))])
def test_strides_of_axes_of_one_element(tokens, n_heads, axes):
    rng = np.random.default_rng(tokens + n_heads)
    c = Case(rng, [20], [tokens], n_heads, 64, 16)
    x = bf16(_block.bits(heads(rng, tokens, n_heads, 64)))
    view = odd(x, axes)
    assert any(s % 8 for s in view.stride()[:2])
    rope, pos = bl.Rope(table(64)), i32(np.arange(20, 20 + tokens))
    say(f"views with strides {view.stride()}")
    want = bl.bl_rope(x, pos, rope)
    out = torch.zeros_like(x)
    bl.bl_rope(view, pos, rope, out=odd(out, axes))
    assert torch.equal(out, want)
    states, outs = [], []
    for t in (x, view):
        cache, batch = c.device()
        q = bl.bl_kv_append(cache, batch, t, t, rope=rope, q=t)
        outs.append((q, bl.bl_attention(cache, batch, t)))
        states.append((cache.k, cache.v, cache.k_absmax, cache.v_absmax))
    assert torch.equal(outs[0][0], want)
    for a, b in zip(outs[0] + states[0], outs[1] + states[1]):
        assert torch.equal(a, b)
