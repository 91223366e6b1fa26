"""The operators together, as examples/decoder_block.py uses them: prompts and
captured single-token steps of a small decoder, and the training gradients of
norm -> BitLinear."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, f32, host, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

_spec = importlib.util.spec_from_file_location(
    "decoder_block", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py"))
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)

SMALL = dict(hidden=256, q_heads=4, kv_heads=2, ffn=320)


def rows(n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((n, SMALL["hidden"]), generator=g, device=DEV).to(torch.bfloat16)


def test_captured_steps_equal_eager_ones():
    lengths, steps = [37, 5, 64], 4
    decoders = [ex.Decoder(2, 3, 80, DEV, page_tokens=16, seed=3, **SMALL) for _ in range(2)]
    prompt = rows(sum(lengths), 4)
    say("decoder: prompt, then captured and eager steps")
    outs = [d.forward(prompt, d.batch([0, 0, 0], lengths)) for d in decoders]
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0].float()).all()
    tokens = [rows(3, 10 + i) for i in range(steps)]
    offsets = torch.arange(4, dtype=torch.int32, device=DEV)
    x, start = tokens[0].clone(), torch.tensor(lengths, dtype=torch.int32, device=DEV)
    graph, row = decoders[0].capture(x, start)
    for i in range(steps):
        # the same bounds as the capture has, so that the same kernels run
        at = torch.tensor([n + i for n in lengths], dtype=torch.int32, device=DEV)
        want = decoders[1].forward(tokens[i], bl.KVBatch(decoders[1].table, at, offsets, 3, 1, 80))
        x.copy_(tokens[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(row, want), f"step {i}"
        assert start.tolist() == [n + i + 1 for n in lengths]
    for a, b in zip(decoders[0].caches, decoders[1].caches):
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.k_absmax, b.k_absmax)


def test_tokens_one_by_one_follow_the_prompt():
    """The same rows as one prompt and one at a time.  The outputs differ by
    roundings of the cache alone: a code that is moved to a grown scale is off
    by up to half a step twice, of values whose size the norms keep near 1.
    With 127 steps to the top and a few such roundings averaged per output,
    5 % of the output's own size is far above what that gives, and far below
    what a wrong position, page or mask does (over 50 %)."""
    n = 40
    d = [ex.Decoder(1, 1, 64, DEV, page_tokens=16, seed=5, **SMALL) for _ in range(2)]
    x = rows(n, 6)
    say("decoder: one prompt against single tokens")
    whole = d[0].forward(x, d[0].batch([0], [n])).float()
    single = torch.cat([d[1].forward(x[i:i + 1], d[1].batch([i], [1])) for i in range(n)]).float()
    assert float((single - whole).norm() / whole.norm()) < 0.05


def test_training_gradients_of_norm_and_layer():
    rng = np.random.default_rng(8)
    m, n, k = 5, 128, 192
    r = _block.bf16_round(rng.standard_normal((m, k)).astype(np.float32))
    w = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
    dy = _block.bf16_round(0.1 * rng.standard_normal((m, n)).astype(np.float32))
    packed, gamma = bl.bl_ternarize_pack(f32((0.02 * rng.standard_normal((n, k))).astype(np.float32)))
    say("norm -> BitLinear backward")
    rd = bf16(_block.bits(r))
    xq, alpha, *_ = bl.bl_rmsnorm_quant(rd, f32(w), ex.EPS)
    dx, dw, dW = ex.norm_linear_backward(bf16(_block.bits(dy)), rd, f32(w), packed, gamma, xq, alpha)
    q = host(bl.bl_unpack_ternary(packed, n, k)).astype(np.float64)
    dn = float(host(gamma)[0]) * dy.astype(np.float64) @ q
    want_dx, want_dw = _block.norm_gradients(dn, r.astype(np.float64), w.astype(np.float64), ex.EPS)
    scale = np.abs(want_dx).max()
    # dn is within (n + 2) 2^-24 of its terms, dx adds bf16's rounding
    assert (np.abs(bf16_bits_to_f64(host(dx)) - want_dx) <= np.abs(want_dx) * _block.U16 + scale * 2.0 ** -14).all()
    assert (np.abs(host(dw) - want_dw) <= np.abs(want_dw).max() * 2.0 ** -14).all()
    xhat = host(xq).astype(np.float64) * host(alpha).astype(np.float64)[:, None] / 127
    want_dW = dy.astype(np.float64).T @ xhat
    # alpha has fp32's bits here: alpha * dy is held as two bf16, right to 2^-17
    terms = np.abs(dy.astype(np.float64)).T @ np.abs(xhat)
    assert (np.abs(host(dW) - want_dW) <= terms * 2.0 ** -17 + terms * (m + 2) * _block.U32).all()
