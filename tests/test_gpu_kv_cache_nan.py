"""NaN and infinities among appended keys and values: they reach their own page
and head and nothing else."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import bf16, say
from test_gpu_kv_cache import Case, heads, table

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


@pytest.mark.parametrize("ctx,new", [([5, 0], [1, 1]), ([9, 3], [40, 20]), ([0, 100], [300, 7])])
@pytest.mark.parametrize("rot", [0, 64, 34])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_appended_value_that_is_not_finite(ctx, new, rot, value):
    rng = np.random.default_rng(sum(new))
    c = Case(rng, ctx, new, 2, 64, 16)
    x = heads(rng, c.total, 4, 64)
    rope = bl.Rope(table(rot)) if rot else None

    def append():
        cache, batch = c.device()
        xd = bf16(_block.bits(x))
        bl.bl_kv_append(cache, batch, xd[:, :2], xd[:, 2:], rope=rope)
        k, v = bl.bl_kv_read(cache, batch)
        return [a.copy() for a in c.state()] + [t.float().cpu().numpy() for t in (k, v)]

    clean = append()
    t = new[0] - 1  # the first sequence's last token
    x[t, 1, 20] = value       # its key, second head
    x[t, 2, 63] = -value      # its value, first head
    say(f"bl_kv_append with {value} ctx={ctx} new={new} rot={rot}")
    got = append()
    page = (ctx[0] + t) // 16
    p, same = c.table[0, page], [i for i in range(c.total) if i >= new[0] or (ctx[0] + i) // 16 != page]
    inside = [i for i in range(new[0]) if i not in same]
    for codes, absmax, back, was, head in ((got[0], got[1], got[4], (clean[0], clean[1], clean[4]), 1),
                                           (got[2], got[3], got[5], (clean[2], clean[3], clean[5]), 0)):
        assert not np.isfinite(absmax[p, head]) and np.isnan(back[inside, head]).all()
        np.testing.assert_array_equal(back[same], was[2][same])
        np.testing.assert_array_equal(back[inside, 1 - head], was[2][inside, 1 - head])
        codes[p, head], absmax[p, head] = was[0][p, head], was[1][p, head]
        np.testing.assert_array_equal(codes, was[0])
        np.testing.assert_array_equal(absmax, was[1])
