"""GPU checks of log probabilities, entropies and alternatives of rows far from 0:
but for lse they do not change with a row's level, so neither do their bounds."""
import numpy as np
import pytest
import torch

import _block
from _gpu import say
from test_gpu_logprobs import check, device, rows

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

LEVELS = [0.0, 30.0, -40.0, 63.0, 65.0, -300.0, 300.0, 505.0, 515.0, -515.0, 30000.0, -1e6, 2.0 ** 23, 2.0 ** 24 + 8, -3e7, 1e9,
          1e20, -1e30, 1e38, -1e38, 3e38]


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("n", [1, 300, 5003, 33000, 70001, 128256])
def test_scores_at_any_level(n, is_bf16):
    rng = np.random.default_rng(n)
    x = rows(rng, len(LEVELS), n, False) + np.asarray(LEVELS, np.float32)[:, None]
    x = _block.bf16_round(x) if is_bf16 else x
    target = rng.integers(n, size=len(LEVELS))
    say(f"bl_logprobs levels n={n} bf16={is_bf16}")
    for scale, top in ((0.7, 0), (0.7, 5), (2.0 ** -20, 1), (1e-3, 0)):
        check(x, device(x, is_bf16), target, scale, top)


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("n", [5003, 70001, 200000])
def test_parts_of_a_row_at_other_levels(n, is_bf16):
    """Masks of every size over whole parts of a row, and levels on either side of those at which the sums are taken
    otherwise."""
    rng = np.random.default_rng(n)
    near, low = 2.0 ** 28 / 1.4426950408889634, float(torch.finfo(torch.bfloat16).min if is_bf16 else torch.finfo(torch.float32).min)
    ends = [(0.0, -1e4), (0.0, -1e9), (0.0, -1e30), (0.0, low), (0.0, -np.inf), (-1e9, low), (near * 1.001, near * 0.999),
            (-near * 1.001, -near * 0.999), (near * 1.1, -near * 1.1), (1e30, 5.0), (-1e30, low), (low, low), (low, -np.inf)]
    x = rows(rng, 2 * len(ends), n, False)
    with np.errstate(invalid="ignore"):
        for i, (a, b) in enumerate(ends):
            cut = int(rng.integers(1, n))
            x[2 * i, :cut], x[2 * i, cut:] = x[2 * i, :cut] + np.float32(a), np.float32(b) if abs(b) > 1e9 else x[2 * i, cut:] + np.float32(b)
            x[2 * i + 1, :cut], x[2 * i + 1, cut:] = np.float32(b), x[2 * i + 1, cut:] + np.float32(a)
    x = _block.bf16_round(x) if is_bf16 else x
    target = rng.integers(n, size=len(x))
    say(f"bl_logprobs parts n={n} bf16={is_bf16}")
    check(x, device(x, is_bf16), target, 1.0, 3)
    check(x, device(x, is_bf16), target, 0.9, 0)
