"""GPU checks of the RMS norm with int8 output and of its gradients against
64-bit references on the same inputs.

Bounds.  n: the fp32 sum h, its square sum (at most 32 additions in a thread,
then a tree) and c are right to about 2^-18 relative, so alpha is too; y adds
bf16's unit 2^-8; a code is within half a step plus 127 * 2^-17 of n * 127 /
alpha; r and xhat are single roundings of known fp32 values (exact bits).
dx: the same relative error on each of its terms plus the bf16 rounding;
dw: fp32 sums, at most (m + 64) roundings.
"""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, f32, host, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

EPS = 1e-5
REL = 2.0 ** -17


def values(rng, m, k, scale=1.0):
    x = rng.standard_normal((m, k)).astype(np.float32) * np.float32(scale)
    x[:, rng.choice(k, size=3)] *= 20
    return _block.bf16_round(x)


@pytest.mark.parametrize("m,k,scale", [
    (1, 64, 1.0), (2, 128, 1e-3), (3, 2048, 1.0), (1, 2112, 1.0), (5, 2560, 30.0), (1, 4096, 1.0), (2, 4160, 1.0),
    (33, 6912, 1.0), (2, 8192, 1.0), (1, 8256, 1.0), (3, 16384, 1.0), (2, 16448, 1.0), (2, 28672, 1.0), (1, 32768, 1e4)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_matches_reference(m, k, scale, residual):
    rng = np.random.default_rng(m * 1000 + k)
    x, w = values(rng, m, k, scale), (1 + 0.3 * rng.standard_normal(k)).astype(np.float32)
    res = values(rng, m, k, 2 * scale) if residual else None
    if m > 1:
        x[1] = 0
        if residual:
            res[1] = 0  # a row of zeros: codes 0, alpha 0
    say(f"bl_rmsnorm_quant m={m} k={k} residual={residual}")
    xq, alpha, r, y, xhat = bl.bl_rmsnorm_quant(
        bf16(_block.bits(x)), f32(w), EPS, residual=bf16(_block.bits(res)) if residual else None, y=True, xhat=True)
    xq, alpha, y, xhat = host(xq), host(alpha), host(y), host(xhat)
    h32 = x + res if residual else x  # one fp32 addition
    if residual:
        np.testing.assert_array_equal(host(r), _block.bits(_block.bf16_round(h32)))
    else:
        assert r is None
    h = x.astype(np.float64) + (res if residual else 0)
    n = _block.norm(h, w.astype(np.float64), EPS)
    top = np.abs(n).max(axis=1)
    assert (np.abs(alpha - top) <= top * REL).all()
    assert (np.abs(bf16_bits_to_f64(y) - n) <= np.abs(n) * (_block.U16 + REL)).all()
    want = n * 127 / np.maximum(top, 1e-5)[:, None]
    assert (np.abs(xq - want) <= 0.5 + 127 * 2 * REL).all()
    assert np.abs(xq.astype(int)).max() <= 127
    step = (alpha / np.float32(127)).astype(np.float32)
    np.testing.assert_array_equal(xhat, _block.bits(_block.bf16_round(xq.astype(np.float32) * step[:, None])))
    if m > 1:
        assert alpha[1] == 0 and (xq[1] == 0).all()


def test_norm_outputs_are_optional_and_in_place():
    rng = np.random.default_rng(3)
    x, res, w = values(rng, 4, 320), values(rng, 4, 320), np.ones(320, np.float32)
    xb, rb, wb = bf16(_block.bits(x)), bf16(_block.bits(res)), f32(w)
    say("bl_rmsnorm_quant optional outputs")
    xq, alpha, r, y, xhat = bl.bl_rmsnorm_quant(xb, wb, EPS, residual=rb, y=True, xhat=True)
    only_y = bl.bl_rmsnorm_quant(xb, wb, EPS, residual=rb, r=False, y=True, xq=False)
    assert only_y[0] is None and only_y[1] is None and only_y[2] is None and torch.equal(only_y[3], y)
    again = bl.bl_rmsnorm_quant(xb, wb, EPS, residual=rb, r=rb)  # the sum replaces the residual
    assert torch.equal(again[0], xq) and torch.equal(again[1], alpha) and torch.equal(rb, r)


def test_norm_feeds_the_product():
    """The codes are what bl_linear takes: the product equals the one from the dequantized rows."""
    rng = np.random.default_rng(4)
    m, n, k = 3, 48, 320
    x, w = values(rng, m, k), np.ones(k, np.float32)
    packed, gamma = bl.bl_ternarize_pack(f32((rng.standard_normal((n, k)) * 0.02).astype(np.float32)))
    say("bl_rmsnorm_quant -> bl_linear")
    xq, alpha, _, _, _ = bl.bl_rmsnorm_quant(bf16(_block.bits(x)), f32(w), EPS)
    acc, y = bl.bl_linear(packed, gamma, xq, alpha, n)
    q = host(bl.bl_unpack_ternary(packed, n, k)).astype(np.int64)
    want = host(xq).astype(np.int64) @ q.T
    np.testing.assert_array_equal(host(acc), want)
    scaled = want * float(host(gamma)[0]) * host(alpha).astype(np.float64)[:, None] / 127
    assert (np.abs(bf16_bits_to_f64(host(y)) - scaled) <= np.abs(scaled) * 2 * _block.U16).all()


@pytest.mark.parametrize("m,k", [(1, 64), (2, 128), (7, 320), (3, 2048), (5, 2560), (600, 192), (1025, 64), (33, 6912),
                                 (4, 8192), (3, 8256), (2, 28672), (513, 4096), (1, 32768)])
@pytest.mark.parametrize("residual", [False, True])
def test_backward_matches_reference(m, k, residual):
    rng = np.random.default_rng(m * 77 + k)
    r, w = values(rng, m, k), (1 + 0.3 * rng.standard_normal(k)).astype(np.float32)
    dn = (0.01 * rng.standard_normal((m, k))).astype(np.float32)
    dr = _block.bf16_round(0.02 * rng.standard_normal((m, k)).astype(np.float32)) if residual else None
    if m > 1:
        r[1] = 0
    say(f"bl_rmsnorm_backward m={m} k={k} residual={residual}")
    args = (f32(dn), bf16(_block.bits(r)), f32(w), EPS)
    dx, dw = bl.bl_rmsnorm_backward(*args, dr=bf16(_block.bits(dr)) if residual else None)
    h, w64, d = r.astype(np.float64), w.astype(np.float64), dn.astype(np.float64)
    want_dx, want_dw = _block.norm_gradients(d, h, w64, EPS)
    c = 1 / np.sqrt((h * h).mean(axis=1, keepdims=True) + EPS)
    terms = c * np.abs(d * w64) + np.abs(h) * c ** 3 * np.abs(d * w64 * h).mean(axis=1, keepdims=True)
    if residual:
        want_dx = want_dx + dr
        terms = terms + np.abs(dr)
    got = bf16_bits_to_f64(host(dx))
    assert (np.abs(got - want_dx) <= np.abs(want_dx) * _block.U16 + terms * REL).all()
    bound = (m + 64) * _block.U32 * np.abs(d * h * c).sum(axis=0) + REL * np.abs(d * h * c).sum(axis=0)
    assert (np.abs(host(dw) - want_dw) <= bound).all()
    again = bl.bl_rmsnorm_backward(*args, dr=bf16(_block.bits(dr)) if residual else None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # fixed order of sums


def test_backward_against_differences_of_the_forward():
    """The kernel's gradients along random directions against central
    differences of the 64-bit forward.  The dw direction is fp32 all the way
    (1e-5); dx carries the bf16 rounding of each element (relative 2^-8 of the
    terms, added in quadrature: 2^-8 * the norm of the terms)."""
    rng = np.random.default_rng(9)
    m, k, step = 6, 192, 1e-4
    r, w = values(rng, m, k).astype(np.float64), 1 + 0.3 * rng.standard_normal(k)
    w = w.astype(np.float32).astype(np.float64)
    dn = rng.standard_normal((m, k)).astype(np.float32)
    say("bl_rmsnorm_backward against differences")
    dx, dw = bl.bl_rmsnorm_backward(f32(dn), bf16(_block.bits(r)), f32(w), EPS)
    dx, dw = bf16_bits_to_f64(host(dx)), host(dw).astype(np.float64)
    loss = lambda a, b: (dn * _block.norm(a, b, EPS)).sum()  # noqa: E731
    for _ in range(5):
        u, v = rng.standard_normal((m, k)), rng.standard_normal(k)
        diff = (loss(r + step * u, w) - loss(r - step * u, w)) / (2 * step)
        assert abs(diff - (dx * u).sum()) <= _block.U16 * np.sqrt(((dx * u) ** 2).sum()) * 4 + 1e-4
        diff = (loss(r, w + step * v) - loss(r, w - step * v)) / (2 * step)
        assert abs(diff - (dw * v).sum()) <= 1e-4 * np.abs(dw * v).sum()


def test_backward_of_no_rows_clears_dw_and_writes_over_dr():
    w = f32(np.ones(64, np.float32))
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device=w.device)
    say("bl_rmsnorm_backward m=0")
    dx, dw = bl.bl_rmsnorm_backward(empty.float(), empty, w, EPS, dw=torch.full((64,), 7.0, device=w.device))
    assert dx.shape == (0, 64) and (host(dw) == 0).all()
    rng = np.random.default_rng(2)
    dn, r, dr = f32(rng.standard_normal((3, 64)).astype(np.float32)), bf16(_block.bits(values(rng, 3, 64))), bf16(_block.bits(values(rng, 3, 64)))
    want, _ = bl.bl_rmsnorm_backward(dn, r, w, EPS, dr=dr)
    bl.bl_rmsnorm_backward(dn, r, w, EPS, dr=dr, dx=dr)
    assert torch.equal(dr, want)


def test_norm_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(12)
    x, w = bf16(_block.bits(values(rng, 9, 2560))), f32(np.ones(2560, np.float32))
    say("bl_rmsnorm_quant on a side stream and captured")
    want = bl.bl_rmsnorm_quant(x, w, EPS)[:2]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = bl.bl_rmsnorm_quant(x, w, EPS)[:2]
        dn = torch.full((9, 2560), 0.5, device=x.device)
        out = [torch.empty_like(t) for t in want]
        grads = (torch.empty_like(x), torch.empty_like(w))
        ws = torch.empty(bl.bl_rmsnorm_backward_workspace_bytes(9, 2560), dtype=torch.uint8, device=x.device)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    eager = bl.bl_rmsnorm_backward(dn, x, w, EPS)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bl.bl_rmsnorm_quant(x, w, EPS, xq=out[0], alpha=out[1])
        bl.bl_rmsnorm_backward(dn, x, w, EPS, dx=grads[0], dw=grads[1], workspace=ws)
    for _ in range(3):
        for t in (*out, *grads, ws):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert torch.equal(grads[0], eager[0]) and torch.equal(grads[1], eager[1])


def test_backward_workspace_on_the_host_is_refused():
    dn, r, w = torch.ones((2, 64), device=DEV), torch.ones((2, 64), dtype=torch.bfloat16, device=DEV), torch.ones(64, device=DEV)
    with pytest.raises(ValueError, match="workspace"):
        bl.bl_rmsnorm_backward(dn, r, w, workspace=torch.empty(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        bl.bl_rmsnorm_backward(dn, r, w, workspace=torch.empty((1 << 16, 2), dtype=torch.uint8, device=DEV)[:, 0])


@pytest.mark.parametrize("m,k", [(259, 6912), (300, 4160), (515, 2048), (1030, 1024), (257, 16384), (258, 12352),
                                 (257, 8256), (259, 16448)])
def test_backward_of_more_rows_than_workgroups(m, k):
    """A workgroup's second row, in each of the kernel's forms."""
    test_backward_matches_reference(m, k, True)
