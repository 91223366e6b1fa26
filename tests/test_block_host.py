"""Host side of the operators around the BitLinear layers: frequency tables,
refusals (every call here is rejected, or has nothing to do, before anything is
enqueued) and the 64-bit reference against itself.  No GPU needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl

BL_OK, BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP = range(6)
FAKE = 0x10000  # aligned, non-null, never dereferenced
lib = bl.library()


def struct(cls, *values):
    s = cls._Struct(*values)
    return s, ctypes.addressof(s)


# ---- frequencies ----

def table_value(rot, **kw):
    t = bl.bl_rope_frequencies(rot, **kw).numpy().astype(np.float64)
    assert t.shape == (rot // 2, 2)
    # value and remainder: the remainder is at most half a unit of the value
    assert (np.abs(t[:, 1]) <= 2.0 ** -24 * np.abs(t[:, 0])).all()
    return t.sum(axis=1)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (96, 500000.0), (256, 10000.0), (34, 1e6)])
def test_plain_and_linear_tables(rot, base):
    want = _block.frequencies(rot, base) / (2 * math.pi)
    # two fp32 hold 48 bits; the 64-bit evaluation of the powers differs by a few units
    np.testing.assert_allclose(table_value(rot, base=base), want, rtol=2.0 ** -45)
    np.testing.assert_allclose(table_value(rot, base=base, scaling="linear", factor=8.0), want / 8, rtol=2.0 ** -45)


def test_base_scaling_slows_the_slowest_pair_by_the_factor_and_not_the_fastest():
    plain, scaled = table_value(64), table_value(64, scaling="base", factor=4.0)
    assert scaled[0] == plain[0]
    assert abs(plain[-1] / scaled[-1] - 4.0) < 1e-9
    assert (np.diff(plain / scaled) > 0).all()


def test_blend_keeps_fast_pairs_and_interpolates_slow_ones():
    kw = dict(factor=8.0, original=8192.0, fast=4.0, slow=1.0)
    plain, got = table_value(128, base=500000.0), table_value(128, base=500000.0, scaling="blend", **kw)
    turns = 8192.0 * plain
    fast, slow = turns >= 4.0, turns <= 1.0
    assert fast.any() and slow.any() and (~fast & ~slow).any()
    np.testing.assert_allclose(got[fast], plain[fast], rtol=2.0 ** -45)
    np.testing.assert_allclose(got[slow], plain[slow] / 8, rtol=2.0 ** -45)
    part = (turns - 1.0) / 3.0
    want = plain * (part + (1 - part) / 8)
    np.testing.assert_allclose(got[~fast & ~slow], want[~fast & ~slow], rtol=1e-12)


def test_frequency_refusals():
    f, out = lib.bl_rope_frequencies, (ctypes.c_float * 256)()
    p = ctypes.addressof(out)
    assert f(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, p) == BL_OK
    assert f(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None) == BL_ERR_NULL
    for rot in (0, -2, 3, 258):
        assert f(rot, 1e4, 0, 1.0, 0.0, 0.0, 0.0, p) == BL_ERR_SHAPE
    for base in (0.0, -1.0, math.inf, math.nan):
        assert f(64, base, 0, 1.0, 0.0, 0.0, 0.0, p) == BL_ERR_SHAPE
    assert f(64, 1e4, 4, 1.0, 0.0, 0.0, 0.0, p) == BL_ERR_SHAPE
    assert f(64, 1e4, 1, 0.0, 0.0, 0.0, 0.0, p) == BL_ERR_SHAPE
    assert f(2, 1e4, 2, 2.0, 0.0, 0.0, 0.0, p) == BL_ERR_SHAPE
    assert f(64, 1e4, 3, 2.0, 0.0, 4.0, 1.0, p) == BL_ERR_SHAPE     # no original length
    assert f(64, 1e4, 3, 2.0, 4096.0, 1.0, 4.0, p) == BL_ERR_SHAPE  # slow >= fast
    with pytest.raises(KeyError):
        bl.bl_rope_frequencies(64, scaling="other")


# ---- refusals ----

def test_rmsnorm_quant_refusals():
    def call(x=FAKE, residual=None, w=FAKE, m=1, k=64, eps=1e-5, r=None, y=None, xhat=None, xq=FAKE, alpha=FAKE):
        return lib.bl_rmsnorm_quant(x, residual, w, m, k, eps, r, y, xhat, xq, alpha, None)

    assert call(x=None) == BL_ERR_NULL
    assert call(w=None) == BL_ERR_NULL
    assert call(xq=None) == BL_ERR_NULL and call(alpha=None) == BL_ERR_NULL  # both or neither
    assert call(xq=None, alpha=None) == BL_ERR_NULL                          # no output at all
    for k in (0, 32, 100, -64, 32768 + 64):
        assert call(k=k) == BL_ERR_SHAPE
    assert call(m=-1) == BL_ERR_SHAPE and call(m=(1 << 23) + 1) == BL_ERR_SHAPE
    for eps in (-1e-5, math.nan, math.inf):
        assert call(eps=eps) == BL_ERR_SHAPE
    for name in ("x", "residual", "w", "r", "y", "xhat", "xq"):
        assert call(**{name: FAKE + 8}) == BL_ERR_ALIGN
    assert call(alpha=FAKE + 2) == BL_ERR_ALIGN
    assert call(m=0, x=None, w=None, xq=None, alpha=None) == BL_OK


def test_rmsnorm_backward_refusals():
    need = bl.bl_rmsnorm_backward_workspace_bytes(3, 64)
    assert need > 0 and bl.bl_rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert bl.bl_rmsnorm_backward_workspace_bytes(3, 65) == 0

    def call(dn=FAKE, r=FAKE, w=FAKE, dr=None, m=3, k=64, eps=1e-5, dx=FAKE, dw=FAKE, ws=FAKE, nbytes=need):
        return lib.bl_rmsnorm_backward(dn, r, w, dr, m, k, eps, dx, dw, ws, nbytes, None)

    for name in ("dn", "r", "w", "dx", "dw", "ws"):
        assert call(**{name: None}) == BL_ERR_NULL
    assert call(k=96) == BL_ERR_SHAPE and call(m=-1) == BL_ERR_SHAPE and call(k=32832) == BL_ERR_SHAPE
    assert call(eps=-1.0) == BL_ERR_SHAPE
    for name in ("dn", "r", "w", "dr", "dx", "ws"):
        assert call(**{name: FAKE + 8}) == BL_ERR_ALIGN
    assert call(dw=FAKE + 2) == BL_ERR_ALIGN
    assert call(nbytes=need - 1) == BL_ERR_WORKSPACE


def test_rope_refusals():
    def call(x=FAKE, xt=128, xh=64, pos=FAKE, turns=FAKE, rot=64, mag=1.0, tokens=1, heads=2, dim=64, y=FAKE, yt=128, yh=64):
        keep, rope = struct(bl.Rope, turns, rot, 0, mag)
        return lib.bl_rope(x, xt, xh, pos, rope, tokens, heads, dim, 0, y, yt, yh, None)

    assert lib.bl_rope(FAKE, 64, 64, FAKE, None, 1, 1, 64, 0, FAKE, 64, 64, None) == BL_ERR_NULL
    for name in ("x", "pos", "turns", "y"):
        assert call(**{name: None}) == BL_ERR_NULL
    for rot in (0, 63, 66, -2):
        assert call(rot=rot) == BL_ERR_SHAPE
    for dim in (0, 60, 264):
        assert call(dim=dim, rot=2) == BL_ERR_SHAPE
    assert call(mag=math.nan) == BL_ERR_SHAPE
    assert call(tokens=-1) == BL_ERR_SHAPE and call(heads=-1) == BL_ERR_SHAPE
    for name in ("x", "y", "turns"):
        assert call(**{name: FAKE + 8}) == BL_ERR_ALIGN
    for name in ("xt", "xh", "yt", "yh"):
        assert call(**{name: 68}) == BL_ERR_ALIGN
    assert call(tokens=0, x=None, pos=None, y=None) == BL_OK
    assert call(heads=0) == BL_OK


CACHE = dict(k=FAKE, v=FAKE, ka=FAKE, va=FAKE, pages=8, heads=2, page=16, dim=64)
BATCH = dict(table=FAKE, start=FAKE, offsets=FAKE, seqs=2, stride=4, tokens=6, max_new=3, max_len=40)


def cache_batch(**kw):
    c, b = dict(CACHE), dict(BATCH)
    for key, value in kw.items():
        (c if key in c else b)[key] = value
    return struct(bl.KVCache, *c.values()), struct(bl.KVBatch, *b.values())


BAD_SHAPES = [dict(heads=0), dict(heads=65537), dict(page=24), dict(page=8), dict(page=512), dict(dim=0), dict(dim=72),
              dict(dim=272), dict(pages=0), dict(pages=1 << 31), dict(seqs=-1), dict(seqs=65536), dict(tokens=-1),
              dict(tokens=(1 << 29) + 1), dict(max_new=-1), dict(max_new=7), dict(max_len=2), dict(max_len=65),
              dict(stride=-1), dict(max_len=(1 << 29) + 1, stride=1 << 30)]
NULLS = ("k", "v", "ka", "va", "table", "start", "offsets")


def check_kv_arguments(call):
    for bad in BAD_SHAPES:
        assert call(**bad) == BL_ERR_SHAPE, bad
    for name in NULLS:
        assert call(**{name: None}) == BL_ERR_NULL, name
        assert call(**{name: FAKE + 2}) == BL_ERR_ALIGN, name
    for name in ("k", "v"):
        assert call(**{name: FAKE + 8}) == BL_ERR_ALIGN, name
    for nothing in (dict(seqs=0), dict(tokens=0, max_new=0), dict(max_new=0)):
        assert call(**nothing) == BL_OK, nothing


def test_kv_append_refusals():
    def call(kk=FAKE, kt=128, kh=64, vv=FAKE, vt=128, vh=64, rot=None, turns=FAKE, q=None, qt=256, qh=64, q_heads=4,
             q_out=None, **kw):
        (c, cp), (b, bp) = cache_batch(**kw)
        keep = rope = None
        if rot is not None:
            keep, rope = struct(bl.Rope, turns, rot, 0, 1.0)
        return lib.bl_kv_append(cp, bp, kk, kt, kh, vv, vt, vh, rope, q, qt, qh, q_heads, q_out, None)

    assert lib.bl_kv_append(None, None, FAKE, 64, 64, FAKE, 64, 64, None, None, 0, 0, 0, None, None) == BL_ERR_NULL
    check_kv_arguments(call)
    assert call(kk=None) == BL_ERR_NULL and call(vv=None) == BL_ERR_NULL
    assert call(rot=64, turns=None) == BL_ERR_NULL
    assert call(q=FAKE, q_out=FAKE) == BL_ERR_NULL          # q is only rotated: no rope
    assert call(q=FAKE, rot=64) == BL_ERR_NULL              # nowhere to write it
    assert call(rot=66) == BL_ERR_SHAPE and call(rot=0) == BL_ERR_SHAPE
    assert call(q=FAKE, q_out=FAKE, rot=64, q_heads=0) == BL_ERR_SHAPE
    for name in ("kk", "vv"):
        assert call(**{name: FAKE + 8}) == BL_ERR_ALIGN
    for name in ("kt", "kh", "vt", "vh"):
        assert call(**{name: 65}) == BL_ERR_ALIGN
    assert call(q=FAKE + 8, q_out=FAKE, rot=64) == BL_ERR_ALIGN
    assert call(q=FAKE, q_out=FAKE + 8, rot=64) == BL_ERR_ALIGN
    assert call(q=FAKE, q_out=FAKE, rot=64, qt=100) == BL_ERR_ALIGN


def test_kv_read_refusals():
    def call(kk=FAKE, vv=FAKE, **kw):
        (c, cp), (b, bp) = cache_batch(**kw)
        return lib.bl_kv_read(cp, bp, kk, vv, None)

    check_kv_arguments(call)
    assert call(kk=None) == BL_ERR_NULL and call(vv=None) == BL_ERR_NULL
    assert call(kk=FAKE + 8) == BL_ERR_ALIGN


def test_attention_refusals():
    def call(q=FAKE, qt=256, qh=64, q_heads=4, scale=0.125, window=0, sinks=0, out=FAKE, lse=None, ws=FAKE,
             nbytes=1 << 40, **kw):
        (c, cp), (b, bp) = cache_batch(**kw)
        return lib.bl_attention(cp, bp, q, qt, qh, q_heads, scale, window, sinks, out, lse, ws, nbytes, None)

    check_kv_arguments(call)
    assert call(q=None) == BL_ERR_NULL and call(out=None) == BL_ERR_NULL
    assert call(q_heads=3) == BL_ERR_SHAPE and call(q_heads=0) == BL_ERR_SHAPE
    for scale in (math.nan, math.inf, -math.inf):
        assert call(scale=scale) == BL_ERR_SHAPE
    assert call(window=-1) == BL_ERR_SHAPE and call(window=8, sinks=-1) == BL_ERR_SHAPE
    assert call(sinks=4) == BL_ERR_SHAPE  # sinks without a window
    assert call(q=FAKE + 8) == BL_ERR_ALIGN and call(out=FAKE + 8) == BL_ERR_ALIGN and call(ws=FAKE + 8) == BL_ERR_ALIGN
    assert call(qt=100) == BL_ERR_ALIGN and call(lse=FAKE + 2) == BL_ERR_ALIGN
    long = dict(pages=4096, stride=2048, max_len=32768, tokens=2, max_new=1)
    (c, cp), (b, bp) = cache_batch(**long)
    need = lib.bl_attention_workspace_bytes(cp, bp, 4)
    assert need > 0
    assert call(nbytes=need - 1, **long) == BL_ERR_WORKSPACE
    assert call(ws=None, **long) == BL_ERR_NULL
    assert lib.bl_attention_workspace_bytes(cp, bp, 3) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((1, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError):
        bl.bl_rmsnorm_quant(x, w)
    with pytest.raises(ValueError):
        bl.bl_rmsnorm_backward(x.float(), x, w)
    with pytest.raises(ValueError):
        bl.Rope(torch.zeros((32, 2)))
    with pytest.raises(ValueError):
        bl.KVCache.empty(4, 2, 16, 64, "cpu")


# ---- the 64-bit reference ----

def test_reference_gradients_agree_with_differences():
    rng = np.random.default_rng(5)
    h, w, dn = rng.standard_normal((3, 64)), 1 + 0.2 * rng.standard_normal(64), rng.standard_normal((3, 64))
    dx, dw = _block.norm_gradients(dn, h, w, 1e-5)
    step = 1e-5  # truncation ~ step^2, rounding ~ 1e-16 / step
    for _ in range(20):
        i, j = rng.integers(3), rng.integers(64)
        e = np.zeros_like(h)
        e[i, j] = step
        diff = ((dn * (_block.norm(h + e, w, 1e-5) - _block.norm(h - e, w, 1e-5))).sum()) / (2 * step)
        assert abs(diff - dx[i, j]) < 1e-8
        e = np.zeros_like(w)
        e[j] = step
        diff = ((dn * (_block.norm(h, w + e, 1e-5) - _block.norm(h, w - e, 1e-5))).sum()) / (2 * step)
        assert abs(diff - dw[j]) < 1e-8


def test_reference_rotation_is_orthogonal_and_relative():
    rng = np.random.default_rng(6)
    x, y = rng.standard_normal((2, 4, 3, 32))
    for interleaved in (False, True):
        f = _block.frequencies(24)
        turned = _block.rotate(x, np.arange(4) + 7, f, interleaved)
        back = _block.rotate(turned, np.arange(4) + 7, f, interleaved, inverse=True)
        np.testing.assert_allclose(back, x, atol=1e-12)
        # q . k depends on the difference of positions alone
        dots = [(_block.rotate(x, np.arange(4) + a, f, interleaved) * _block.rotate(y, np.arange(4) + a + 3, f, interleaved)).sum(-1)
                for a in (0, 50)]
        np.testing.assert_allclose(dots[0], dots[1], atol=1e-12)
