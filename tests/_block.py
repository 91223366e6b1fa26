"""Plain 64-bit implementations of the operators around the BitLinear layers
(norm, rotary positions, 8-bit cache, attention), on numpy arrays, and the
error bounds that the formulas give.  No code of the package is used."""
from __future__ import annotations

import numpy as np

U16 = 2.0 ** -8   # unit roundoff of bf16
U32 = 2.0 ** -24  # of fp32


def bf16_round(a: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest, ties to even), as fp32."""
    b = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).reshape(np.shape(a))


def bits(a: np.ndarray) -> np.ndarray:
    """bf16 bit patterns of values that are bf16 already."""
    return (np.ascontiguousarray(a, np.float32).view(np.uint32) >> 16).astype(np.uint16)


# ---- norm ----

def norm(h, w, eps):
    """n = h * w / sqrt(mean h^2 + eps), rows of a 64-bit array."""
    return h * w / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)


def norm_gradients(dn, h, w, eps):
    """(dx, dw) of sum(dn * norm(h, w)) by the quotient rule."""
    k = h.shape[1]
    v = (h * h).mean(axis=1, keepdims=True) + eps
    g = dn * w
    return g / np.sqrt(v) - h * (g * h).sum(axis=1, keepdims=True) / (k * v ** 1.5), (dn * h / np.sqrt(v)).sum(axis=0)


# ---- rotary positions ----

def frequencies(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)


def rotate(x, pos, freq, interleaved=False, inverse=False, magnitude=1.0):
    """[tokens][heads][dim] rotated over its first 2 * len(freq) elements."""
    y, half = np.array(x, np.float64), len(freq)
    angle = (np.asarray(pos, np.float64)[:, None] * freq)[:, None] * (-1.0 if inverse else 1.0)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    z = (y[..., first] + 1j * y[..., second]) * (magnitude * np.exp(1j * angle))
    y[..., first], y[..., second] = z.real, z.imag
    return y


def rotation_bound(x, freq, interleaved, magnitude):
    """Largest |output| of each element's pair: what errors of cos and sin multiply."""
    y, half = np.abs(np.array(x, np.float64)), len(freq)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    both = magnitude * (y[..., first] + y[..., second])
    y[..., first], y[..., second] = both, both
    return y


# The fraction of a turn is right to about 2^-23 turns = 7.5e-7 rad, the
# hardware's cos and sin and three fp32 roundings add the rest.
ANGLE = 2.0 ** -16


# ---- cache ----

def append(codes, absmax, table, start, offsets, x):
    """The cache after new rows x (fp32 [tokens][heads][dim]) entered, by the
    fp32 arithmetic that the header states."""
    codes, absmax = codes.copy(), absmax.copy()
    pages, heads, page, _ = codes.shape
    f = np.float32
    for s in range(len(start)):
        a, n = int(start[s]), int(offsets[s + 1] - offsets[s])
        at = a // page * page if n else a
        while at < a + n:
            p = table[s][at // page]
            keep, end = max(0, a - at), min(page, a + n - at)
            rows = x[offsets[s] + at + keep - a:offsets[s] + at + end - a]
            if 0 <= p < pages:
                for h in range(heads):
                    old = absmax[p, h] if keep else f(0)
                    top = f(max(old, np.abs(rows[:, h]).max()))
                    if top < 2.0 ** -64:
                        top = f(0)
                    if keep and top > old:
                        codes[p, h, :keep] = np.rint(codes[p, h, :keep].astype(f) * f(old / top)).astype(np.int8)
                    scale = f(f(127) / top) if top > 0 else f(0)
                    codes[p, h, keep:end] = np.rint(rows[:, h].astype(f) * scale).astype(np.int8)
                    absmax[p, h] = top
            at += page
    return codes, absmax


def read(codes, absmax, table, start, offsets):
    """bf16 values (as fp32) of the batch's tokens."""
    pages, heads, page, dim = codes.shape
    out = np.zeros((int(offsets[-1]), heads, dim), np.float32)
    for s in range(len(start)):
        for i in range(int(offsets[s + 1] - offsets[s])):
            pos = int(start[s]) + i
            p = table[s][pos // page]
            if 0 <= p < pages:
                step = (absmax[p].astype(np.float32) / np.float32(127)).astype(np.float32)
                out[offsets[s] + i] = bf16_round(codes[p, :, pos % page].astype(np.float32) * step[:, None])
    return out


# ---- attention ----

def attention(q, k_codes, k_absmax, v_codes, v_absmax, table, start, offsets, scale, window=0, sinks=0):
    """(out, lse, bound of |error of out| before its rounding, bound of lse's) in 64 bits.

    The bound: a query element is off by at most absmax / 65024, so a score by
    that times scale * sum |k|, and fp32 evaluation adds a few units of 2^-24 of
    the base-2 exponents involved; a weight's relative error is at most delta +
    2^-11 (fp16), once above and once below the fraction; below fp16's normal
    range a weight is off by at most 2^-39 of the row's largest p * absmax."""
    pages, heads, page, dim = k_codes.shape
    tokens, q_heads, _ = q.shape
    group = q_heads // heads
    out, bound = np.zeros((tokens, q_heads, dim)), np.zeros((tokens, q_heads, dim))
    lse, lse_bound = np.full((tokens, q_heads), -np.inf), np.zeros((tokens, q_heads))
    for s in range(len(start)):
        a, n = int(start[s]), int(offsets[s + 1] - offsets[s])
        if n == 0:
            continue
        ids = np.asarray([table[s][i] for i in range((a + n + page - 1) // page)])
        there = (ids >= 0) & (ids < pages)
        safe = np.where(there, ids, 0)
        key = np.arange(a + n)
        at = (a + np.arange(n))[:, None]
        seen = (key <= at) & np.repeat(there, page)[:a + n]
        if window:
            seen &= (at - key < window) | (key < sinks)
        for h in range(heads):
            def values(codes, top):
                step = np.where(there, top[safe, h].astype(np.float64), 0.0) / 127.0
                return (codes[safe, h].astype(np.float64) * step[:, None, None]).reshape(-1, dim)[:a + n]
            k, v = values(k_codes, k_absmax), values(v_codes, v_absmax)
            for g in range(group):
                rows = q[offsets[s]:offsets[s] + n, h * group + g].astype(np.float64)
                score = np.where(seen, scale * (rows @ k.T), -np.inf)
                top = score.max(axis=1, keepdims=True)
                e = np.exp(score - np.where(np.isfinite(top), top, 0.0))
                total = e.sum(axis=1, keepdims=True)
                p = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
                here = (slice(offsets[s], offsets[s] + n), h * group + g)
                out[here] = p @ v
                with np.errstate(divide="ignore"):
                    lse[here] = (np.log(total) + top)[:, 0]
                off = abs(scale) * np.abs(rows).max(axis=1) / 65024.0 * np.abs(k).sum(axis=1).max()
                finite = np.where(seen, np.abs(score, where=seen, out=np.zeros_like(score)), 0.0).max(axis=1)
                delta = off + 8 * U32 * (finite + 64.0)
                largest = (p * np.repeat(np.where(there, np.abs(v_absmax[safe, h]), 0.0), page)[:a + n]).max(axis=1)
                bound[here] = (2 * delta + 2.0 ** -10)[:, None] * (p @ np.abs(v)) + (2.0 ** -39 * largest * seen.sum(axis=1))[:, None]
                lse_bound[here] = delta + 2.0 ** -18
    return out, lse, bound, lse_bound
