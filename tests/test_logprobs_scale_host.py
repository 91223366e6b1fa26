"""Scales of the log probabilities on the host: those whose product with log2 e
is past fp32 are refused.  No GPU needed."""
import numpy as np
import pytest

import ternary_weight_absmean_amd as bl
from test_block_host import BL_ERR_NULL, BL_ERR_SHAPE, FAKE

lib = bl.library()


@pytest.mark.parametrize("scale,status", [(2.0 ** 127, BL_ERR_NULL), (float(np.nextafter(np.float32(2.0 ** 127), np.float32(np.inf))), BL_ERR_SHAPE),
                                          (3e38, BL_ERR_SHAPE), (1e-45, BL_ERR_NULL)])
def test_scales(scale, status):
    """A scale that is taken gets as far as the missing logits."""
    assert lib.bl_logprobs(None, 0, 3, 100, 100, scale, None, 0, None, FAKE, None, None, None, None, 0, None) == status
    assert lib.bl_logprobs_backward(None, 0, 3, 100, 100, scale, None, FAKE, None, None, None, FAKE, FAKE, 100, None) == status
