"""Plain implementations of the operators for many answers to one prompt (pages
of the cache on Python lists, log probabilities on numpy arrays in 64 bits) and
the error bounds that the formulas give.  No code of the package is used."""
from __future__ import annotations

import numpy as np

from _block import U16, U32


# ---- pages ----

class Pool:
    """refs, and the calls that change them; tables are lists of rows."""

    def __init__(self, refs, page):
        self.refs, self.page = list(refs), page

    def there(self, e):
        return 0 <= e < len(self.refs)

    def lowest(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def release(self, e):
        if self.there(e) and self.refs[e] > 0:
            self.refs[e] -= 1

    def grow(self, table, start, count, copies=None):
        short, free, left = 0, self.lowest()[::-1], []
        for row, a, n in zip(table, start, count):
            a = max(a, 0)
            if copies is not None:
                copies.append((-1, -1, 0))
            if n <= 0:
                continue
            for i in range(a // self.page, (a + n - 1) // self.page + 1):
                shared = copies is not None and i * self.page < a and i < len(row) and self.there(row[i])
                if shared and self.refs[row[i]] - left.count(row[i]) > 1:
                    if free:  # a sequence that gets no page goes on holding the shared one
                        left.append(row[i])
                        copies[-1] = (row[i], free.pop(), a % self.page)
                        row[i] = copies[-1][1]
                        self.refs[row[i]] = 1
                    else:
                        copies[-1] = (row[i], -1, 0)
                        short += 1
                elif i < len(row) and not self.there(row[i]):
                    if free:
                        row[i] = free.pop()
                        self.refs[row[i]] = 1
                    else:
                        short += 1
        for e in left:
            self.release(e)
        return short

    def fork(self, table, length, parent, keep):
        stride = len(table[0]) if table else 0
        free, short = self.lowest()[::-1], 0
        out, out_length, copies, elder = [], [], [], set()
        gone = [list(r) for r in table]
        for p in parent:
            row, n, copy = [-1] * stride, 0, (-1, -1, 0)
            if 0 <= p < len(table):
                n = min(max(length[p], 0), stride * self.page)
                full, rest = divmod(n, self.page)
                first = not keep and p not in elder
                elder.add(p)
                for i in range(full):
                    row[i] = table[p][i]
                    if first:
                        gone[p][i] = -1
                    elif self.there(row[i]):
                        self.refs[row[i]] += 1
                if rest and self.there(table[p][full]):
                    if first:
                        row[full], gone[p][full] = table[p][full], -1
                    elif free:
                        row[full] = free.pop()
                        self.refs[row[full]] = 1
                        copy = (table[p][full], row[full], rest)
                    else:
                        short += 1
            out.append(row)
            out_length.append(n)
            copies.append(copy)
        if not keep:
            for r in gone:
                for e in r:
                    self.release(e)
        return out, out_length, copies, short

    def free(self, table, keep=None):
        for s, row in enumerate(table):
            n = max(keep[s], 0) if keep is not None else 0
            for i in range(-(-n // self.page), len(row)):
                self.release(row[i])
                row[i] = -1

    def compact(self, table, moves):
        used = [p for p, r in enumerate(self.refs) if r]
        n = len(used)
        above, below = [p for p in used if p >= n][::-1], [p for p in range(n) if not self.refs[p]]
        pairs = list(zip(above, below))[:moves]
        name = dict(pairs)
        for a, b in pairs:
            self.refs[b], self.refs[a] = self.refs[a], 0
        for row in table:
            row[:] = [name.get(e, e) for e in row]
        return [(a, b, self.page) for a, b in pairs] + [(-1, -1, 0)] * (moves - len(pairs)), len(pairs)


def copy_pages(k, absmax, copies):
    """[pages][heads][page][dim] codes and [pages][heads] scales after the copies."""
    k, absmax = k.copy(), absmax.copy()
    for a, b, n in copies:
        if 0 <= a < len(k) and 0 <= b < len(k) and n > 0:
            k[b, :, :n] = k[a, :, :n]
            absmax[b] = absmax[a]
    return k, absmax


# ---- log probabilities ----

def logprobs(x, target, scale=1.0, top=0):
    """Dictionary of the outputs of rows x, and bounds of their errors, in 64 bits.

    The kernel's d_j = (x_j - max) scale log2 e takes four roundings, so it is off by 4 units of itself; a sum of n
    terms goes through at most 65 additions in a thread and 20 across threads, exp2 and log2 are right to
    two units: relative to S at most (4 sum p_j |d_j| + 90) units, and alike for W = sum e d with d once more."""
    x = np.asarray(x, np.float64)
    m, n = x.shape
    with np.errstate(all="ignore"):
        most = x.max(axis=1)
        base = np.where(np.isneginf(most), 0.0, most)
        d = (x - base[:, None]) * scale
        e = np.exp(d)
        s = e.sum(axis=1)
        lse = base * scale + np.log(s)
        p = np.divide(e, s[:, None], out=np.zeros_like(e), where=s[:, None] != 0)
        far = np.where(e > 0, -d, 0.0)
        entropy = np.where(s == 0, 0.0, np.log(s) + (p * far).sum(axis=1))
        log_p = np.where(np.isneginf(x) & ~np.isnan(s)[:, None], -np.inf, d - np.log(s)[:, None])
    lse = np.where(s == 0, -np.inf, lse)
    mean_far, square = (p * far).sum(axis=1), (p * far * far).sum(axis=1)
    log_s = np.abs(np.log(np.where(s > 0, s, 1.0)))
    of_sum = U32 * (8 * mean_far + 8 * log_s + 128)
    out = {"lse": lse, "entropy": entropy, "log_p": log_p, "p": p, "sum_bound": of_sum,
           "lse_bound": of_sum + U32 * 4 * np.abs(np.where(np.isfinite(lse), lse, 0.0)),
           "entropy_bound": of_sum + U32 * (16 * square + 256 * mean_far)}
    if target is not None:
        t = np.asarray(target)
        known = (t >= 0) & (t < n)
        safe = np.where(known, t, 0)
        out["logprob"] = np.where(known, log_p[np.arange(m), safe], 0.0)
    if top:
        ids, values = np.full((m, top), -1), np.full((m, top), -np.inf)
        for i in range(m):
            real = np.where(x[i] > -np.inf)[0]  # no NaN among them
            order = real[np.lexsort((real, -x[i, real]))][:top]
            ids[i, :len(order)], values[i, :len(order)] = order, log_p[i, order]
        out["top_id"], out["top_logprob"] = ids, values
    return out


def logprob_bound(value, of_sum):
    """Of a log probability: its own d and logarithm beside the sum's."""
    return of_sum[:, None] + 16 * U32 * (np.abs(np.where(np.isfinite(value), value, 0.0)) + 16)


def logprobs_gradient(x, target, g=None, gh=None, gz=None, scale=1.0, bf16=False):
    """(gradient, bound of its error) for lse and entropy as the kernel gives them."""
    m, n = x.shape
    zero = np.zeros(m)
    g, gh, gz = (zero if v is None else np.asarray(v, np.float64) for v in (g, gh, gz))
    r = logprobs(x, None, scale)
    p, entropy = r["p"], r["entropy"][:, None]
    log_p = np.where(p > 0, r["log_p"], 0.0)
    t = np.full(m, -1) if target is None else np.asarray(target)
    known = (t >= 0) & (t < n)
    g = np.where(known, g, 0.0)[:, None]
    gh, gz = gh[:, None], gz[:, None]
    hit = np.zeros((m, n))
    hit[np.arange(m)[known], t[known]] = 1.0
    want = scale * (g * (hit - p) + gz * p - gh * p * (log_p + entropy))
    none = (np.isneginf(r["lse"])[:, None]) | ((g == 0) & (gh == 0) & (gz == 0))
    want = np.where(none, 0.0, want)
    lse = np.where(np.isfinite(r["lse"]), r["lse"], 0.0)[:, None]
    # a weight's relative error: lse's, the roundings of z - lse and of the exponential
    off = r["lse_bound"][:, None] + U32 * (2 * np.abs(lse) + 8 * np.abs(log_p) + 8)
    size = np.abs(g) + np.abs(gz) + np.abs(gh) * (np.abs(log_p) + entropy)
    bound = scale * p * (size * (off + 8 * U32) + np.abs(gh) * (r["entropy_bound"][:, None] + off)) + 4 * U32 * scale * np.abs(g) * hit
    bound = np.where(none, 0.0, bound)
    return want, bound + (U16 if bf16 else U32) * (np.abs(want) + bound) + 2.0 ** -120
