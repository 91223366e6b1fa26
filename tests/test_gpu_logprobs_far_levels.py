"""GPU checks of log probabilities and their gradient on either side of the level
(2^30 in base 2) from which on only a row's largest elements count, and of masks
past it over whole parts of rows."""
import numpy as np
import pytest
import torch

import _block
from _gpu import f32, say
from test_gpu_logprobs import check, device, rows
from test_gpu_logprobs_gradient_levels import check_gradient

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

LEVELS = [1e8, 1.5e8, -1.8e8, 3e8, -5e8, 7e8, -7.4e8, 7.45e8, 1e9, -1.2e9, 1.45e9, 1.5e9, -2e9, 2.2e9, 3.1e9, 5e9, -7e9, 1e12, 1e29, 1e31]


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1.3])
@pytest.mark.parametrize("n", [1, 2, 300, 5003, 70001])
def test_levels_around_the_far_one(n, scale, is_bf16):
    """Logits as they come, and all within a few units in the last place of each other."""
    rng = np.random.default_rng(n)
    level = np.asarray(LEVELS, np.float32)[:, None]
    x = rows(rng, len(LEVELS), n, False) + level
    steps = rng.integers(0, 4, size=x.shape)
    if is_bf16:  # 2^16 fp32 units to one of bf16
        bits = _block.bf16_round(np.broadcast_to(level, x.shape).astype(np.float32)).view(np.int32) - (steps << 16)
    else:
        bits = np.broadcast_to(level, x.shape).astype(np.float32).view(np.int32) - steps
    x = np.concatenate([_block.bf16_round(x) if is_bf16 else x, bits.astype(np.int32).view(np.float32)])
    target = rng.integers(n, size=len(x))
    say(f"bl_logprobs around the far level n={n} scale={scale} bf16={is_bf16}")
    xd = device(x, is_bf16)
    scale = float(np.float32(scale))
    check(x, xd, target, scale, 0)
    _, lse, entropy, _, _ = check(x, xd, target, scale, min(n, 3))
    g, gh, gz = rng.standard_normal((3, len(x))).astype(np.float32)
    check_gradient(x, xd, target, lse, entropy, (g, gh, gz), scale, is_bf16)


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("mask", [-1e9, -7.4e8, -7.5e8, -1e30, -3e38])
def test_masks_over_parts_of_rows(mask, is_bf16):
    rng = np.random.default_rng(7)
    n = 128256
    x = rows(rng, 8, n, False)
    for i, cut in enumerate((0, 1, 20000, 50000, 64128, 100000, n - 1, n)):
        x[i, cut:] = mask
    x = _block.bf16_round(x) if is_bf16 else x
    target = rng.integers(n, size=8)
    say(f"bl_logprobs mask={mask} bf16={is_bf16}")
    xd = device(x, is_bf16)
    for top in (0, 20):
        _, lse, entropy, _, _ = check(x, xd, target, 1.0, top)
    g, gh, gz = rng.standard_normal((3, 8)).astype(np.float32)
    check_gradient(x, xd, target, lse, entropy, (g, gh, gz), 1.0, is_bf16)
