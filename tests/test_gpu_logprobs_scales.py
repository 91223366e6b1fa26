"""GPU checks of log probabilities at scales and logits near the ends of fp32's
range: what the products with scale keep finite is right."""
import numpy as np
import pytest
import torch

import _block
from _gpu import say
from test_gpu_logprobs import check, device
from test_gpu_logprobs_gradient_levels import check_gradient

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("n", [7, 3000, 70001])
@pytest.mark.parametrize("power", [-124, -120, -100, -40, 60, 100, 120, 127])
def test_scales_and_logits_of_any_size(power, n, is_bf16):
    """Logits of 2^-power times numbers up to 4 (up to fp32's range), so that their differences may pass it."""
    rng = np.random.default_rng(n + 200 - power)
    z = np.clip(rng.standard_normal((4, n)) * 2, -3.9, 3.9)
    z[1] *= 20
    z[:, 1] = -3.9
    x = np.clip(z * 2.0 ** -power, -3.3e38, 3.3e38).astype(np.float32)
    x = _block.bf16_round(x) if is_bf16 else x
    target = np.array([1, 1, n - 1, 3])
    say(f"bl_logprobs scale 2^{power} n={n} bf16={is_bf16}")
    xd = device(x, is_bf16)
    scale = 2.0 ** power
    _, lse, entropy, _, _ = check(x, xd, target, scale, 6)
    g, gh, gz = (rng.standard_normal((3, 4)) * 2.0 ** min(0, 20 - power)).astype(np.float32)
    check_gradient(x, xd, target, lse, entropy, (g, gh, gz), scale, is_bf16)
