"""Host side of the operators for many answers to one prompt: refusals (every
call here is rejected, or has nothing to do, before anything is enqueued) and
the 64-bit references against themselves.  No GPU needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

import _answers
import ternary_weight_absmean_amd as bl
from test_block_host import (BL_ERR_ALIGN, BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_WORKSPACE, BL_OK, CACHE, FAKE, cache_batch,
                             check_kv_arguments, struct)

lib = bl.library()


def pool(refs=FAKE, pages=100, page=16):
    return struct(bl.KVPool, refs, pages, page)


def check_pool(call):
    for bad in (dict(pages=0), dict(pages=(1 << 24) + 1), dict(page=0), dict(page=24), dict(page=512)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    assert call(refs=None) == BL_ERR_NULL
    assert call(refs=FAKE + 4) == BL_ERR_ALIGN


def test_kv_grow_refusals():
    def call(refs=FAKE, pages=100, page=16, copies=None, shortage=None, **kw):
        keep, pp = pool(refs, pages, page)
        (c, cp), (b, bp) = cache_batch(**kw)
        return lib.bl_kv_grow(pp, bp, copies, shortage, None)

    assert lib.bl_kv_grow(None, None, None, None, None) == BL_ERR_NULL
    check_pool(call)
    for bad in (dict(seqs=-1), dict(seqs=65536), dict(tokens=-1), dict(max_new=-1), dict(max_new=7), dict(max_len=2),
                dict(max_len=65), dict(stride=-1), dict(stride=1 << 26), dict(tokens=(1 << 29) + 1),
                dict(seqs=60000, tokens=1 << 14, max_new=1 << 14, max_len=1 << 14, stride=1 << 10),
                dict(seqs=8193, copies=FAKE)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    for name in ("table", "start", "offsets"):
        assert call(**{name: None}) == BL_ERR_NULL
        assert call(**{name: FAKE + 2}) == BL_ERR_ALIGN
    assert call(copies=FAKE + 2) == BL_ERR_ALIGN and call(shortage=FAKE + 2) == BL_ERR_ALIGN
    for nothing in (dict(seqs=0), dict(tokens=0, max_new=0), dict(max_new=0)):
        assert call(refs=None, table=None, **nothing) == BL_OK


def test_kv_fork_refusals():
    def call(refs=FAKE, pages=100, page=16, table=FAKE, stride=4, length=FAKE, seqs=2, parent=FAKE, children=3, keep=0,
             out=2 * FAKE, out_length=4 * FAKE, copies=FAKE, shortage=None):
        held, pp = pool(refs, pages, page)
        return lib.bl_kv_fork(pp, table, stride, length, seqs, parent, children, keep, out, out_length, copies, shortage, None)

    assert lib.bl_kv_fork(None, FAKE, 4, FAKE, 2, FAKE, 3, 0, FAKE, FAKE, FAKE, None, None) == BL_ERR_NULL
    check_pool(call)
    for bad in (dict(seqs=-1), dict(seqs=8193), dict(children=-1), dict(children=8193), dict(stride=-1), dict(stride=1 << 26),
                dict(out=FAKE), dict(out_length=FAKE)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    for name in ("table", "length", "parent", "out", "out_length", "copies"):
        assert call(**{name: None}) == BL_ERR_NULL, name
        assert call(**{name: 3 * FAKE + 2}) == BL_ERR_ALIGN, name
    assert call(shortage=FAKE + 2) == BL_ERR_ALIGN
    assert call(children=0, keep=1, refs=None) == BL_OK and call(children=0, seqs=0, refs=None) == BL_OK
    assert call(children=0, stride=0, table=None) == BL_OK


def test_kv_free_refusals():
    def call(refs=FAKE, pages=100, page=16, table=FAKE, stride=4, seqs=2, keep=None):
        held, pp = pool(refs, pages, page)
        return lib.bl_kv_free(pp, table, stride, seqs, keep, None)

    assert lib.bl_kv_free(None, FAKE, 4, 2, None, None) == BL_ERR_NULL
    check_pool(call)
    for bad in (dict(seqs=-1), dict(seqs=65536), dict(stride=-1), dict(stride=1 << 26)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    assert call(table=None) == BL_ERR_NULL
    assert call(table=FAKE + 2) == BL_ERR_ALIGN and call(keep=FAKE + 2) == BL_ERR_ALIGN
    assert call(seqs=0, table=None) == BL_OK and call(stride=0, table=None) == BL_OK


def test_kv_compact_refusals():
    held, pp = pool()
    need = lib.bl_kv_compact_workspace_bytes(pp, 50)
    assert need > 0 and lib.bl_kv_compact_workspace_bytes(pp, 101) == 0 and lib.bl_kv_compact_workspace_bytes(pp, -1) == 0
    assert lib.bl_kv_compact_workspace_bytes(None, 1) == 0

    def call(refs=FAKE, pages=100, page=16, table=FAKE, stride=4, seqs=2, moves=50, copies=FAKE, moved=FAKE, ws=FAKE, nbytes=need):
        keep, p = pool(refs, pages, page)
        return lib.bl_kv_compact(p, table, stride, seqs, moves, copies, moved, ws, nbytes, None)

    check_pool(call)
    for bad in (dict(seqs=-1), dict(stride=-1), dict(moves=-1), dict(moves=101)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    for name in ("table", "copies", "moved", "ws"):
        assert call(**{name: None}) == BL_ERR_NULL, name
        assert call(**{name: FAKE + 2}) == BL_ERR_ALIGN, name
    assert call(ws=FAKE + 8) == BL_ERR_ALIGN
    assert call(nbytes=need - 1) == BL_ERR_WORKSPACE


def test_kv_copy_refusals():
    def call(count=2, copies=FAKE, n=3, valid=None, second=None, **kw):
        values = dict(CACHE, **kw)
        other = dict(values, **(second or {}))
        arr = (bl.KVCache._Struct * 2)(bl.KVCache._Struct(*values.values()), bl.KVCache._Struct(*other.values()))
        return lib.bl_kv_copy(ctypes.addressof(arr), count, copies, n, valid, None)

    for bad in (dict(count=-1), dict(count=1025), dict(n=-1), dict(n=(1 << 24) + 1), dict(heads=0), dict(page=24), dict(dim=72),
                dict(pages=0), dict(second=dict(pages=9)), dict(second=dict(heads=1)), dict(second=dict(page=32)),
                dict(second=dict(dim=128))):
        assert call(**bad) == BL_ERR_SHAPE, bad
    assert lib.bl_kv_copy(None, 1, FAKE, 1, None, None) == BL_ERR_NULL
    assert call(copies=None) == BL_ERR_NULL
    for name in ("k", "v", "ka", "va"):
        assert call(**{name: None}) == BL_ERR_NULL and call(second={name: None}) == BL_ERR_NULL
        assert call(**{name: FAKE + 2}) == BL_ERR_ALIGN and call(second={name: FAKE + 2}) == BL_ERR_ALIGN
    assert call(copies=FAKE + 2) == BL_ERR_ALIGN and call(valid=FAKE + 2) == BL_ERR_ALIGN
    assert call(n=0, copies=None) == BL_OK and call(count=0, copies=None) == BL_OK


def test_attention_shared_refusals():
    shared = dict(group=FAKE, prefix=FAKE, groups=2, max_group=1, max_prefix=32)

    def args(kw):
        s = dict(shared)
        for key in list(kw):
            if key in s:
                s[key] = kw.pop(key)
        return cache_batch(**kw), struct(bl.KVShared, *s.values())

    def call(q=FAKE, qt=256, qh=64, q_heads=4, scale=0.125, out=FAKE, lse=None, ws=FAKE, nbytes=1 << 40, **kw):
        ((c, cp), (b, bp)), (s, sp) = args(kw)
        return lib.bl_attention_shared(cp, bp, sp, q, qt, qh, q_heads, scale, out, lse, ws, nbytes, None)

    check_kv_arguments(call)
    (c, cp), (b, bp) = cache_batch()
    assert lib.bl_attention_shared(cp, bp, None, FAKE, 256, 64, 4, 0.125, FAKE, None, FAKE, 1 << 40, None) == BL_ERR_NULL
    for bad in (dict(groups=1), dict(groups=-1), dict(max_group=0), dict(max_group=-1), dict(groups=65536), dict(max_group=65536),
                dict(max_prefix=-1), dict(max_prefix=41), dict(q_heads=3), dict(q_heads=0), dict(scale=math.nan),
                dict(heads=65536, q_heads=65536, tokens=1 << 18, max_new=1, max_len=64),
                dict(scale=math.inf)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    for name in ("q", "out", "group", "prefix"):
        assert call(**{name: None}) == BL_ERR_NULL, name
        assert call(**{name: FAKE + 2}) == BL_ERR_ALIGN, name
    assert call(ws=FAKE + 2) == BL_ERR_ALIGN
    for name in ("q", "out", "ws"):
        assert call(**{name: FAKE + 8}) == BL_ERR_ALIGN, name
    assert call(qt=100) == BL_ERR_ALIGN and call(lse=FAKE + 2) == BL_ERR_ALIGN
    long = dict(pages=4096, stride=2048, seqs=40, tokens=40, max_new=1, max_len=32768, max_group=20, max_prefix=32000)
    ((c, cp), (b, bp)), (s, sp) = args(dict(long))
    need = lib.bl_attention_shared_workspace_bytes(cp, bp, sp, 4)
    assert need > 0 and call(nbytes=need - 1, **long) == BL_ERR_WORKSPACE
    assert call(ws=None, **long) == BL_ERR_NULL
    assert need != lib.bl_attention_workspace_bytes(cp, bp, 4)  # the prefixes are taken together
    assert lib.bl_attention_shared_workspace_bytes(cp, bp, sp, 3) == 0
    # a short prefix is not: what bl_attention needs
    ((c, cp), (b, bp)), (s, sp) = args(dict(long, max_prefix=128))
    assert lib.bl_attention_shared_workspace_bytes(cp, bp, sp, 4) == lib.bl_attention_workspace_bytes(cp, bp, 4)


def test_logprobs_refusals():
    def call(x=FAKE, kind=0, m=3, n=1000, stride=1000, scale=1.0, target=FAKE, top=5, logprob=FAKE, lse=FAKE, entropy=FAKE,
             top_id=FAKE, top_logprob=FAKE, ws=FAKE, nbytes=1 << 40):
        return lib.bl_logprobs(x, kind, m, n, stride, scale, target, top, logprob, lse, entropy, top_id, top_logprob, ws, nbytes,
                               None)

    for bad in (dict(kind=2), dict(kind=-1), dict(m=-1), dict(m=(1 << 23) + 1), dict(n=0), dict(n=(1 << 20) + 1, stride=1 << 21),
                dict(stride=999), dict(m=1 << 23, stride=1 << 18), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
                dict(scale=math.inf), dict(top=-1), dict(top=65)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    for name in ("x", "target", "top_id", "top_logprob"):
        assert call(**{name: None}) == BL_ERR_NULL, name
    assert call(logprob=None, lse=None, entropy=None, top=0) == BL_ERR_NULL
    assert call(x=FAKE + 1) == BL_ERR_ALIGN and call(x=FAKE + 2, kind=1) == BL_ERR_ALIGN
    for name in ("target", "logprob", "lse", "entropy", "top_id", "top_logprob", "ws"):
        assert call(**{name: FAKE + 2}) == BL_ERR_ALIGN, name
    assert call(ws=FAKE + 8) == BL_ERR_ALIGN
    need = bl.bl_logprobs_workspace_bytes(3, 100000, torch.bfloat16, 5)
    assert need > 0
    assert call(n=100000, stride=100000, nbytes=need - 1) == BL_ERR_WORKSPACE
    assert call(n=100000, stride=100000, ws=None) == BL_ERR_NULL
    assert call(m=0, x=None, target=None, logprob=None, top_id=None) == BL_OK
    assert bl.bl_logprobs_workspace_bytes(0, 100, torch.float32, 0) == 0
    assert bl.bl_logprobs_workspace_bytes(1, 100, torch.float32, 65) == 0


def test_logprobs_backward_refusals():
    def call(x=FAKE, kind=0, m=3, n=1000, stride=1000, scale=1.0, target=FAKE, lse=FAKE, entropy=FAKE, g=FAKE, gh=FAKE, gz=FAKE,
             dx=2 * FAKE, dx_stride=1000):
        return lib.bl_logprobs_backward(x, kind, m, n, stride, scale, target, lse, entropy, g, gh, gz, dx, dx_stride, None)

    for bad in (dict(kind=2), dict(m=-1), dict(n=0), dict(stride=999), dict(dx_stride=999), dict(scale=0.0), dict(scale=math.nan),
                dict(dx=FAKE, dx_stride=1001)):
        assert call(**bad) == BL_ERR_SHAPE, bad
    for name in ("x", "target", "lse", "entropy", "dx"):
        assert call(**{name: None}) == BL_ERR_NULL, name
    assert call(g=None, gh=None, gz=None) == BL_ERR_NULL
    for name in ("target", "lse", "entropy", "g", "gh", "gz"):
        assert call(**{name: FAKE + 2}) == BL_ERR_ALIGN, name
    assert call(x=FAKE + 1) == BL_ERR_ALIGN and call(dx=FAKE + 2, kind=1) == BL_ERR_ALIGN
    assert call(m=0, x=None, lse=None, g=None, gh=None, gz=None) == BL_OK


def test_binding_refuses_host_tensors():
    refs = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        bl.KVPool(refs, 16)
    with pytest.raises(ValueError):
        bl.KVPool.empty(8, 16, "cpu")
    with pytest.raises(ValueError):
        bl.KVShared(refs, refs, 1, 1)
    x = torch.zeros((2, 50), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bl.bl_logprobs(x)
    with pytest.raises(ValueError):
        bl.bl_logprobs_backward(x, None, torch.zeros(2), None, None, dlse=torch.zeros(2))


# ---- the references ----

def test_reference_gradient_agrees_with_differences():
    rng = np.random.default_rng(5)
    m, n, scale = 3, 40, 0.7
    x, target = 2 * rng.standard_normal((m, n)), np.array([4, 39, -1])
    x[1, 7] = -np.inf
    g, gh, gz = rng.standard_normal((3, m))

    def total(x):
        r = _answers.logprobs(x, target, scale)
        return (g * r["logprob"] + gh * r["entropy"] + gz * r["lse"]).sum()

    grad, _ = _answers.logprobs_gradient(x, target, g, gh, gz, scale)
    step = 1e-5  # truncation ~ step^2, rounding ~ 1e-16 / step
    for i in range(m):
        for j in range(0, n, 3):
            if not np.isfinite(x[i, j]):
                continue
            e = np.zeros_like(x)
            e[i, j] = step
            assert abs((total(x + e) - total(x - e)) / (2 * step) - grad[i, j]) < 1e-8


def test_reference_statistics_of_simple_rows():
    r = _answers.logprobs(np.zeros((1, 8)), [3], 2.0, 3)
    assert abs(r["entropy"][0] - math.log(8)) < 1e-15 and abs(r["lse"][0] - math.log(8)) < 1e-15
    assert r["top_id"].tolist() == [[0, 1, 2]] and abs(r["logprob"][0] + math.log(8)) < 1e-15
    r = _answers.logprobs(np.array([[-np.inf, 5.0, -np.inf]]), [0], 1.0, 2)
    assert r["entropy"][0] == 0 and r["lse"][0] == 5 and r["logprob"][0] == -np.inf
    assert r["top_id"].tolist() == [[1, -1]] and r["top_logprob"][0].tolist() == [0.0, -np.inf]


def test_reference_pool_gives_back_what_it_gave():
    rng = np.random.default_rng(2)
    pool = _answers.Pool([0] * 60, 16)
    table, length = [[-1] * 6 for _ in range(3)], [0, 0, 0]
    for _ in range(30):
        new = rng.integers(0, 9, size=3).tolist()
        new = [n if a + n < 90 else 0 for a, n in zip(length, new)]
        copies = []
        assert pool.grow(table, length, new, copies) == 0
        length = [a + n for a, n in zip(length, new)]
        table, length, _, short = pool.fork(table, length, rng.integers(3, size=3).tolist(), False)
        assert short == 0
        length = [int(rng.integers(n // 2, n + 1)) for n in length]
        pool.free(table, length)
        pool.compact(table, int(rng.integers(20)))
        held = [e for r in table for e in r if e >= 0]
        assert sum(pool.refs) == len(held) and all(pool.refs[e] == held.count(e) for e in held)
    pool.free(table)
    assert sum(pool.refs) == 0
