"""GPU checks of the RMS norm and its gradients without an eps: rows of zeros
among others, in each of the kernels' forms.  Bounds as in test_gpu_norm.py."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import bf16, bf16_bits_to_f64, f32, host, say
from test_gpu_norm import REL, values

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

SIZES = [(3, 64), (4, 1024), (3, 2048), (5, 2560), (4, 8192), (3, 16384), (3, 32768)]


@pytest.mark.parametrize("m,k", SIZES)
def test_rows_of_zeros_without_an_eps(m, k):
    rng = np.random.default_rng(k)
    x, w = values(rng, m, k), (1 + 0.3 * rng.standard_normal(k)).astype(np.float32)
    x[1] = 0
    say(f"bl_rmsnorm_quant eps=0 m={m} k={k}")
    xq, alpha, _, y, xhat = (t if t is None else host(t) for t in
                             bl.bl_rmsnorm_quant(bf16(_block.bits(x)), f32(w), 0.0, y=True, xhat=True))
    assert alpha[1] == 0 and not xq[1].any() and not (y[1] & 0x7FFF).any() and not (xhat[1] & 0x7FFF).any()
    others = np.arange(m) != 1
    n = _block.norm(x[others].astype(np.float64), w.astype(np.float64), 0.0)
    top = np.abs(n).max(axis=1)
    assert (np.abs(alpha[others] - top) <= top * REL).all()
    assert (np.abs(bf16_bits_to_f64(y[others]) - n) <= np.abs(n) * (_block.U16 + REL)).all()
    assert (np.abs(xq[others] - n * 127 / top[:, None]) <= 0.5 + 127 * 2 * REL).all()


@pytest.mark.parametrize("m,k", SIZES)
def test_gradients_of_rows_of_zeros_without_an_eps(m, k):
    rng = np.random.default_rng(k + 1)
    r, w = values(rng, m, k), (1 + 0.3 * rng.standard_normal(k)).astype(np.float32)
    r[1] = 0
    dn = rng.standard_normal((m, k)).astype(np.float32)
    dr = _block.bf16_round(rng.standard_normal((m, k)).astype(np.float32))
    say(f"bl_rmsnorm_backward eps=0 m={m} k={k}")
    dx, dw = bl.bl_rmsnorm_backward(f32(dn), bf16(_block.bits(r)), f32(w), 0.0, dr=bf16(_block.bits(dr)))
    np.testing.assert_array_equal(host(dx)[1], _block.bits(dr)[1])  # what passes the norm, and nothing through it
    others = np.arange(m) != 1
    h, w64, d = r[others].astype(np.float64), w.astype(np.float64), dn[others].astype(np.float64)
    want_dx, want_dw = _block.norm_gradients(d, h, w64, 0.0)
    c = 1 / np.sqrt((h * h).mean(axis=1, keepdims=True))
    terms = c * np.abs(d * w64) + np.abs(h) * c ** 3 * np.abs(d * w64 * h).mean(axis=1, keepdims=True) + np.abs(dr[others])
    want_dx = want_dx + dr[others]
    assert (np.abs(bf16_bits_to_f64(host(dx))[others] - want_dx) <= np.abs(want_dx) * _block.U16 + terms * REL).all()
    bound = ((m + 64) * _block.U32 + REL) * np.abs(d * h * c).sum(axis=0)
    assert (np.abs(host(dw) - want_dw) <= bound).all()
