"""GPU checks of the rotary positions and of the 8-bit key/value cache.

Codes and absmax of values (not rotated) are exact bits of the stated fp32
arithmetic; rotated values are within the rounding of bf16 (2^-8) plus the
angle's error (2^-16 of the pair's magnitude), rotated keys within half a step
plus the same error."""
import numpy as np
import pytest
import torch

import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, f32, host, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def heads(rng, *shape):
    return _block.bf16_round(rng.standard_normal(shape).astype(np.float32) * np.float32(2))


def table(rot, **kw):
    return bl.bl_rope_frequencies(rot, **kw).to(DEV)


# ---- rotary positions ----

@pytest.mark.parametrize("tokens,n_heads,dim,rot,first", [
    (1, 25, 128, 128, 1234), (1, 1, 8, 2, 0), (3, 2, 64, 64, 5), (7, 3, 80, 80, 100), (5, 4, 96, 48, 4000), (4, 2, 64, 34, 9),
    (2, 3, 56, 56, 70000), (3, 5, 256, 256, 131000), (6, 1, 40, 20, 3), (2, 2, 72, 72, 16000000), (1100, 20, 128, 96, 120000),
    (2, 2, 24, 24, -50)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_reference(tokens, n_heads, dim, rot, first, interleaved, inverse):
    rng = np.random.default_rng(tokens + dim + rot)
    x, pos = heads(rng, tokens, n_heads, dim), first + rng.permutation(tokens)
    mag = 1.0 if dim != 96 else 1.25
    say(f"bl_rope tokens={tokens} heads={n_heads} dim={dim} rot={rot} interleaved={interleaved} inverse={inverse}")
    rope = bl.Rope(table(rot), interleaved=interleaved, magnitude=mag)
    xb = bf16(_block.bits(x))
    out = bl.bl_rope(xb, i32(pos), rope, inverse=inverse)
    freq = _block.frequencies(rot)
    want = _block.rotate(x, pos, freq, interleaved, inverse, mag)
    bound = _block.U16 * np.abs(want) + _block.ANGLE * _block.rotation_bound(x, freq, interleaved, mag)
    got = bf16_bits_to_f64(host(out))
    assert (np.abs(got - want) <= bound).all()
    np.testing.assert_array_equal(host(out)[..., rot:], _block.bits(x)[..., rot:])  # passes unchanged
    bl.bl_rope(xb, i32(pos), rope, inverse=inverse, out=xb)  # in place
    assert torch.equal(xb, out)


def test_rope_on_strided_heads():
    rng = np.random.default_rng(8)
    whole = bf16(_block.bits(heads(rng, 6, 9, 64)))
    q, k = whole[:, :5], whole[:, 5:7]  # as they lie in one projection's output
    pos, rope = i32(np.arange(6) + 11), bl.Rope(table(64))
    say("bl_rope strided")
    want = bl.bl_rope(k.contiguous(), pos, rope)
    rest = whole.clone()
    bl.bl_rope(k, pos, rope, out=k)
    assert torch.equal(k, want)
    assert torch.equal(q, rest[:, :5]) and torch.equal(whole[:, 7:], rest[:, 7:])
    by_head = bf16(_block.bits(heads(rng, 3, 6, 64)))  # [heads][tokens][dim]
    got = bl.bl_rope(by_head.transpose(0, 1), pos, rope)
    assert torch.equal(got, bl.bl_rope(by_head.transpose(0, 1).contiguous(), pos, rope))
    assert bl.bl_rope(whole[:0], i32([]), rope).shape == (0, 9, 64)


def test_rope_gradient_against_differences():
    """sum(dy * rope(x)) has the inverse rotation of dy as its gradient: along a
    random direction the rotation is linear, so the difference is exact."""
    rng = np.random.default_rng(13)
    x, dy, u = (heads(rng, 5, 2, 64) for _ in range(3))
    pos, freq = np.arange(5) + 77, _block.frequencies(64)
    say("bl_rope gradient")
    dx = bf16_bits_to_f64(host(bl.bl_rope(bf16(_block.bits(dy)), i32(pos), bl.Rope(table(64)), inverse=True)))
    loss = lambda a: (dy * _block.rotate(a, pos, freq)).sum()  # noqa: E731
    diff = (loss(x + 0.5 * u) - loss(x - 0.5 * u))
    assert abs(diff - (dx * u).sum()) <= 4 * _block.U16 * np.sqrt(((dx * u) ** 2).sum())


# ---- cache ----

class Case:
    """A cache with earlier tokens in it and a step of new ones."""

    def __init__(self, rng, ctx, new, n_heads=2, dim=64, page=16, spare=3):
        self.rng, self.ctx, self.new, self.page = rng, ctx, new, page
        need = [-(-(a + n) // page) for a, n in zip(ctx, new)]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.table = np.full((len(ctx), max(max(need), 1)), -1)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.k, self.v = (rng.integers(-127, 128, (pages, n_heads, page, dim)).astype(np.int8) for _ in range(2))
        self.ka, self.va = (rng.uniform(0.5, 4, (pages, n_heads)).astype(np.float32) for _ in range(2))
        self.start, self.offsets = np.array(ctx), np.concatenate([[0], np.cumsum(new)])
        self.total = int(self.offsets[-1])
        self.pos = np.concatenate([np.arange(a, a + n) for a, n in zip(ctx, new)] + [np.zeros(0, int)])

    def device(self):
        t = lambda a: torch.from_numpy(a.copy()).to(DEV)  # noqa: E731
        self.cache = bl.KVCache(t(self.k), t(self.v), t(self.ka), t(self.va))
        self.batch = self.step(self.start, self.offsets)
        return self.cache, self.batch

    def step(self, start, offsets):
        lengths = np.diff(offsets)
        return bl.KVBatch(i32(self.table), i32(start), i32(offsets), int(offsets[-1]), int(lengths.max(initial=0)),
                          int((start + lengths).max(initial=0)))

    def state(self):
        return tuple(host(t) for t in (self.cache.k, self.cache.k_absmax, self.cache.v, self.cache.v_absmax))


STEPS = [([0], [1]), ([5], [1]), ([16], [1]), ([15, 31, 0, 7], [1, 1, 1, 1]), ([0], [40]), ([9, 0, 33], [40, 3, 0]),
         ([3, 100, 17], [8, 9, 70]), ([250], [300])]


@pytest.mark.parametrize("ctx,new", STEPS)
@pytest.mark.parametrize("n_heads,dim,page", [(2, 64, 16), (1, 128, 64), (3, 80, 32), (5, 16, 128), (1, 256, 256)])
def test_append_without_rotation_is_exact(ctx, new, n_heads, dim, page):
    rng = np.random.default_rng(sum(ctx) + 31 * sum(new) + dim)
    c = Case(rng, ctx, new, n_heads, dim, page)
    cache, batch = c.device()
    k, v = heads(rng, c.total, n_heads, dim), heads(rng, c.total, n_heads, dim)
    if c.total > 2:
        k[c.total // 2] *= 16  # a late token that raises its page's scale
    k = _block.bf16_round(k)
    say(f"bl_kv_append ctx={ctx} new={new} heads={n_heads} dim={dim} page={page}")
    assert bl.bl_kv_append(cache, batch, bf16(_block.bits(k)), bf16(_block.bits(v))) is None
    kc, ka = _block.append(c.k, c.ka, c.table, c.start, c.offsets, k)
    vc, va = _block.append(c.v, c.va, c.table, c.start, c.offsets, v)
    for got, want in zip(c.state(), (kc, ka, vc, va)):
        np.testing.assert_array_equal(got, want)
    bl.bl_kv_append(cache, batch, bf16(_block.bits(k)), bf16(_block.bits(v)))  # the same tokens again
    for got, want in zip(c.state(), (kc, ka, vc, va)):
        np.testing.assert_array_equal(got, want)
    # the whole of every sequence read back
    lengths = np.array(ctx) + np.array(new)
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    rk, rv = bl.bl_kv_read(cache, c.step(np.zeros(len(ctx), int), offsets))
    start = np.zeros(len(ctx), int)
    np.testing.assert_array_equal(host(rk), _block.bits(_block.read(kc, ka, c.table, start, offsets)))
    np.testing.assert_array_equal(host(rv), _block.bits(_block.read(vc, va, c.table, start, offsets)))


@pytest.mark.parametrize("ctx,new", [([0], [1]), ([70], [1]), ([9, 0, 33], [40, 3, 0]), ([120000], [20])])
@pytest.mark.parametrize("dim,rot,page", [(64, 64, 16), (128, 96, 64), (80, 80, 32), (48, 34, 16), (64, 10, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_with_rotation(ctx, new, dim, rot, page, interleaved):
    rng = np.random.default_rng(sum(ctx) + dim + rot)
    n_heads, q_heads = 2, 6
    c = Case(rng, ctx, new, n_heads, dim, page)
    cache, batch = c.device()
    qkv = heads(rng, c.total, q_heads + 2 * n_heads, dim)
    qkv_d = bf16(_block.bits(qkv))
    q, k, v = qkv_d.split([q_heads, n_heads, n_heads], dim=1)  # strided
    say(f"bl_kv_append rotated ctx={ctx} new={new} dim={dim} rot={rot} page={page} interleaved={interleaved}")
    q_out = bl.bl_kv_append(cache, batch, k, v, rope=bl.Rope(table(rot), interleaved=interleaved), q=q)
    freq = _block.frequencies(rot)
    # q: the same as bl_rope, bit for bit
    want_q = bl.bl_rope(q.contiguous(), i32(c.pos), bl.Rope(table(rot), interleaved=interleaved))
    assert torch.equal(q_out, want_q)
    k64 = _block.rotate(qkv[:, q_heads:q_heads + n_heads], c.pos, freq, interleaved)
    slack = _block.ANGLE * _block.rotation_bound(qkv[:, q_heads:q_heads + n_heads], freq, interleaved, 1.0)
    kc, ka, vc, va = c.state()
    want_vc, want_va = _block.append(c.v, c.va, c.table, c.start, c.offsets, qkv[:, q_heads + n_heads:])
    np.testing.assert_array_equal(vc, want_vc)
    np.testing.assert_array_equal(va, want_va)
    for s, (a, n) in enumerate(zip(ctx, new)):
        for i in range(n):
            p, slot, t = c.table[s, (a + i) // page], (a + i) % page, c.offsets[s] + i
            step = ka[p].astype(np.float64)[:, None] / 127
            # half a step and the angle's error; the top value may exceed absmax by that error alone
            assert (np.abs(kc[p, :, slot] * step - k64[t]) <= step * (0.5 + 2.0 ** -12) + slack[t]).all()
            assert (np.abs(k64[t]).max(axis=1) <= ka[p] + slack[t].max(axis=1)).all()


def test_append_to_missing_pages_writes_nothing_there():
    rng = np.random.default_rng(21)
    c = Case(rng, [10, 0], [30, 20])
    c.table[0, 1], c.table[1, 0] = -1, 10 ** 6  # neither is a page
    cache, batch = c.device()
    k, v = heads(rng, 50, 2, 64), heads(rng, 50, 2, 64)
    say("bl_kv_append missing pages")
    bl.bl_kv_append(cache, batch, bf16(_block.bits(k)), bf16(_block.bits(v)))
    kc, ka = _block.append(c.k, c.ka, c.table, c.start, c.offsets, k)
    vc, va = _block.append(c.v, c.va, c.table, c.start, c.offsets, v)
    for got, want in zip(c.state(), (kc, ka, vc, va)):
        np.testing.assert_array_equal(got, want)
    rk, _ = bl.bl_kv_read(cache, batch, k=torch.full((50, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV))
    want = _block.read(kc, ka, c.table, c.start, c.offsets)
    assert (want[6:22] == 0).all()
    np.testing.assert_array_equal(host(rk) & 0x7FFF, _block.bits(want) & 0x7FFF)


def test_append_of_zeros_and_of_tiny_values():
    rng = np.random.default_rng(22)
    c = Case(rng, [0, 0, 5], [4, 4, 2])
    cache, batch = c.device()
    v = heads(rng, 10, 2, 64)
    v[0:4] = 0
    v[4:8] *= np.float32(2.0 ** -80)  # below the smallest absmax that is kept
    v[8:10] = 0                       # a page that has earlier tokens keeps its scale
    say("bl_kv_append zeros")
    bl.bl_kv_append(cache, batch, bf16(_block.bits(v)), bf16(_block.bits(v)))
    vc, va = _block.append(c.v, c.va, c.table, c.start, c.offsets, v)
    _, _, got_c, got_a = c.state()
    np.testing.assert_array_equal(got_c, vc)
    np.testing.assert_array_equal(got_a, va)
    assert (got_a[c.table[0, 0]] == 0).all() and (got_a[c.table[1, 0]] == 0).all() and (got_a[c.table[2, 0]] > 0).all()


def test_append_in_two_steps_equals_the_reference_in_two_steps():
    """Token by token into the same page: scales only grow, earlier codes follow."""
    rng = np.random.default_rng(23)
    c = Case(rng, [0], [24], n_heads=1)
    cache, _ = c.device()
    x = heads(rng, 24, 1, 64) * np.float32(2) ** np.arange(24)[:, None, None].astype(np.float32)
    x = _block.bf16_round(x)
    kc, ka = c.k, c.ka
    say("bl_kv_append token by token")
    for i in range(24):
        b = c.step(np.array([i]), np.array([0, 1]))
        one = bf16(_block.bits(x[i:i + 1]))
        bl.bl_kv_append(cache, b, one, one)
        kc, ka = _block.append(kc, ka, c.table, np.array([i]), np.array([0, 1]), x[i:i + 1])
    got = c.state()
    np.testing.assert_array_equal(got[0], kc)
    np.testing.assert_array_equal(got[1], ka)
