"""GPU checks of the cosine and sine of the rotary positions to fp32's precision.

Rotated keys show them before any rounding to bf16: a page's absmax is the fp32
maximum over its keys.  A key whose only pair is (1, 0) gives max(|cos|, |sin|),
(1, 1) gives |cos| + |sin|.  Bounds: the reduced angle f (below an eighth of a
turn) and the remainder added to it are rounded once each to 2^-28 turns (4.7e-8
rad together); 2 pi in fp32, its polynomial and the product add 2.8e-8 + 2 * 2^-25
relative to at most 0.71, the cosine's last two steps 2^-25 + 0.3 * 2^-24: 2^-23 in
all.  The sum of two is off by twice that and its own rounding."""
import numpy as np
import pytest
import torch

import ternary_weight_absmean_amd as bl
from _gpu import DEV, host, say
from test_gpu_kv_cache import i32

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

PAGE = 16


def absmax_of_rotated_keys(turns, pos, pair, interleaved, dim):
    """[positions][pairs]: one sequence with a page of its own per position, one head per pair."""
    n, pairs = len(pos), turns.shape[0]
    k = torch.zeros((n, pairs, dim), dtype=torch.bfloat16, device=DEV)
    at = torch.arange(pairs, device=DEV)
    first, second = (2 * at, 2 * at + 1) if interleaved else (at, at + pairs)
    k[:, at, first], k[:, at, second] = pair
    cache = bl.KVCache.empty(n, pairs, PAGE, dim, DEV)
    table = torch.full((n, int(pos.max()) // PAGE + 1), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(n, device=DEV), torch.from_numpy(pos // PAGE).to(DEV)] = torch.arange(n, dtype=torch.int32, device=DEV)
    batch = bl.KVBatch(table, i32(pos), i32(np.arange(n + 1)), n, 1, int(pos.max()) + 1)
    bl.bl_kv_append(cache, batch, k, k, rope=bl.Rope(turns.to(DEV), interleaved=interleaved))
    return host(cache.k_absmax).astype(np.float64)


@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 34)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,top", [(1024, 1 << 10), (1024, 1 << 14), (24, 1 << 24)])
def test_cosine_and_sine_are_right_to_fp32(dim, rot, interleaved, n, top):
    rng = np.random.default_rng(top + rot)
    pos = np.arange(n) if top == n else np.sort(rng.choice(top, n, replace=False))
    turns = bl.bl_rope_frequencies(rot)
    t = turns.numpy().astype(np.float64).sum(axis=1)
    p = pos[:, None] * t
    angle = 2 * np.pi * (p - np.rint(p))
    c, s = np.abs(np.cos(angle)), np.abs(np.sin(angle))
    say(f"bl_kv_append: cosine and sine dim={dim} rot={rot} interleaved={interleaved} positions below {top}")
    one = absmax_of_rotated_keys(turns, pos, (1.0, 0.0), interleaved, dim)
    assert np.abs(one - np.maximum(c, s)).max() <= 2.0 ** -23
    both = absmax_of_rotated_keys(turns, pos, (1.0, 1.0), interleaved, dim)
    assert np.abs(both - (c + s)).max() <= 2 * 2.0 ** -23 + 2.0 ** -24
