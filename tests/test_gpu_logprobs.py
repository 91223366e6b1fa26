"""GPU checks of log probabilities, entropy, alternatives and their gradient
against 64-bit evaluations; bounds as derived in _answers."""
import numpy as np
import pytest
import torch

import _answers
import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, f32, host, say

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

INF = np.inf


def rows(rng, m, n, is_bf16):
    """Logits as a vocabulary's product gives them, and as the device takes them."""
    x = (2.0 * rng.standard_normal((m, n))).astype(np.float32)
    for i in range(m):
        x[i, rng.integers(n, size=min(n, 6))] += rng.uniform(0, 12)
    return _block.bf16_round(x) if is_bf16 else x


def device(x, is_bf16, lead=0, pad=0):
    """x as a view inside a wider buffer of NaNs (lead elements before each row, pad after)."""
    m, n = x.shape
    wide = np.full((m, lead + n + pad), np.nan, np.float32)
    wide[:, lead:lead + n] = x
    t = bf16(_block.bits(wide)) if is_bf16 else f32(wide)
    return t[:, lead:lead + n]


def f64(t):
    return bf16_bits_to_f64(host(t)) if t.dtype == torch.bfloat16 else host(t).astype(np.float64)


def near(got, want, bound):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want) - bound
    bad = ~same & ~(off <= 0)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside their bound: {got[bad][:4]} for {want[bad][:4]}"


def check(x, xd, target, scale=1.0, top=0):
    scale = float(np.float32(scale))
    want = _answers.logprobs(x, target, scale, top)
    td = torch.from_numpy(np.asarray(target, np.int32)).to(DEV)
    got = bl.bl_logprobs(xd, td, scale=scale, top=top)
    near(f64(got[0]), want["logprob"], _answers.logprob_bound(want["logprob"][:, None], want["sum_bound"])[:, 0])
    near(f64(got[1]), want["lse"], want["lse_bound"])
    near(f64(got[2]), want["entropy"], want["entropy_bound"])
    if top:
        assert np.array_equal(host(got[3]), want["top_id"])
        near(f64(got[4]), want["top_logprob"], _answers.logprob_bound(want["top_logprob"], want["sum_bound"]))
    again = bl.bl_logprobs(xd, td, scale=scale, top=top)
    for a, b in zip(got, again):
        assert a is b is None or torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    return got


SHAPES = [(1, 1, 1), (1, 7, 2), (3, 8, 20), (2, 100, 5), (5, 1000, 64), (1, 4096, 20), (2, 4097, 1), (3, 32769, 20),
          (1, 128256, 20), (7, 50001, 5), (70, 5003, 3), (600, 2000, 20), (40, 40000, 33), (1, 1 << 20, 64)]


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("m,n,top", SHAPES)
def test_matches_reference(m, n, top, is_bf16):
    rng = np.random.default_rng(m * 7 + n + top)
    x = rows(rng, m, n, is_bf16)
    target = rng.integers(n, size=m)
    say(f"bl_logprobs m={m} n={n} top={top} bf16={is_bf16}")
    check(x, device(x, is_bf16), target, 1.0, top)
    check(x, device(x, is_bf16), target, 0.6, 0)


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("lead,pad", [(0, 1), (1, 0), (3, 2), (7, 8), (8, 8), (5, 300)])
@pytest.mark.parametrize("m,n", [(5, 1001), (3, 12), (2, 33000), (4, 3)])
def test_rows_at_any_alignment(m, n, lead, pad, is_bf16):
    """What lies between the rows is NaN and does not matter; a gradient leaves it as it is."""
    rng = np.random.default_rng(n + lead + 10 * pad)
    x = rows(rng, m, n, is_bf16)
    target = rng.integers(n, size=m)
    say(f"bl_logprobs alignment m={m} n={n} lead={lead} pad={pad} bf16={is_bf16}")
    xd = device(x, is_bf16, lead, pad)
    _, lse, entropy, _, _ = check(x, xd, target, 1.3, min(n, 9))
    g, gh = rng.standard_normal((2, m)).astype(np.float32)
    want, bound = _answers.logprobs_gradient(x, target, g, gh, None, float(np.float32(1.3)), is_bf16)
    td = torch.from_numpy(target.astype(np.int32)).to(DEV)
    for other in (pad, pad + 1):  # rows that begin as those of x do, and others
        whole = torch.full((m, lead + n + other), 5.0, dtype=xd.dtype, device=DEV)
        dx = bl.bl_logprobs_backward(xd, td, lse, entropy, f32(g), f32(gh), scale=1.3, dlogits=whole[:, lead:lead + n])
        near(f64(dx), want, bound)
        assert (whole[:, :lead] == 5.0).all() and (whole[:, lead + n:] == 5.0).all()


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("n", [60, 3000, 70000])
def test_masked_rows(n, is_bf16):
    rng = np.random.default_rng(n)
    x = rows(rng, 9, n, is_bf16)
    low = float(torch.finfo(torch.bfloat16).min) if is_bf16 else float(np.finfo(np.float32).min)
    x[0] = -INF                                   # nothing can occur
    x[1] = -INF
    x[1, n // 2] = 3.0                            # one token can
    x[2, rng.random(n) < 0.99] = -INF
    x[3, rng.random(n) < 0.9] = low               # a mask of the type's lowest value
    x[4] = low                                    # nothing but it: all alike
    x[5, :n // 2] = -INF
    x[6] = 0.25                                   # all alike
    x[7] = np.sort(x[7])                          # the largest at the end
    x[8, ::2], x[8, 1::2] = 0.0, -0.0             # equal, of either sign
    target = np.array([3, n // 2, 5, 7, 9, 11, n - 1, n - 1, 0])
    say(f"bl_logprobs masked n={n} bf16={is_bf16}")
    xd = device(x, is_bf16)
    for top in (0, 1, 20, 64):
        got = check(x, xd, target, 1.0, top)
    g, gh, gz = (rng.standard_normal((3, 9)) * 0.1).astype(np.float32)
    want, bound = _answers.logprobs_gradient(x, target, g, gh, gz, 1.0, is_bf16)
    dx = bl.bl_logprobs_backward(xd, torch.from_numpy(target.astype(np.int32)).to(DEV), got[1], got[2], f32(g), f32(gh), f32(gz))
    near(f64(dx), want, bound)
    cannot = np.isneginf(x[2]) & (np.arange(n) != target[2])  # a target's own 1 stays where it cannot occur
    assert (f64(dx)[0] == 0).all() and (f64(dx)[2][cannot] == 0).all()


@pytest.mark.parametrize("is_bf16", [True, False])
def test_nan_and_infinity_stay_in_their_rows(is_bf16):
    rng = np.random.default_rng(5)
    x = rows(rng, 6, 5000, is_bf16)
    clean = x.copy()
    x[1, 77] = np.nan
    x[2, 4999] = INF
    x[3] = np.nan
    x[4, [1, 2]] = INF
    target = np.array([1, 2, 4999, 4, 1, 6])
    say(f"bl_logprobs NaN bf16={is_bf16}")
    xd = device(x, is_bf16)
    td = torch.from_numpy(target.astype(np.int32)).to(DEV)
    got = [host(t) for t in bl.bl_logprobs(xd, td, top=8)]
    plain = [host(t) for t in bl.bl_logprobs(device(clean, is_bf16), td, top=8)]
    for a, b in zip(got, plain):
        assert np.array_equal(a[[0, 5]], b[[0, 5]])
    for k in (0, 1, 2):
        assert np.isnan(got[k][1:5]).all()
    assert np.isnan(got[4][[1, 2, 4]]).all()
    want = _answers.logprobs(np.where(np.isnan(x), -INF, x), None, 1.0, 8)["top_id"]
    assert np.array_equal(got[3], want)
    g = f32(np.ones(6))
    dx = f64(bl.bl_logprobs_backward(xd, td, f32(got[1]), f32(got[2]), g))
    assert np.isnan(dx[1:5]).all() and np.isfinite(dx[[0, 5]]).all()
    # rows without a gradient give zeros whatever they hold
    g[1:5] = 0.0
    dx = f64(bl.bl_logprobs_backward(xd, td, f32(got[1]), f32(got[2]), g))
    assert (dx[1:5] == 0).all() and (dx[0] != 0).any()


def test_targets_outside_the_vocabulary():
    rng = np.random.default_rng(6)
    x = rows(rng, 5, 3000, True)
    target = np.array([-1, 3000, -100, 7, 2 ** 31 - 1])
    say("bl_logprobs targets")
    xd = device(x, True)
    got = check(x, xd, target)
    assert (host(got[0])[[0, 1, 2, 4]] == 0).all()
    g, gz = rng.standard_normal((2, 5)).astype(np.float32)
    want, bound = _answers.logprobs_gradient(x, target, g, None, gz, 1.0, True)
    dx = bl.bl_logprobs_backward(xd, torch.from_numpy(target.astype(np.int32)).to(DEV), got[1], None, f32(g), None, f32(gz))
    near(f64(dx), want, bound)


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("m,n", [(1, 1), (3, 700), (2, 33001), (300, 515)])
def test_gradient_matches_formula(m, n, is_bf16):
    rng = np.random.default_rng(m + n)
    x = rows(rng, m, n, is_bf16)
    target = rng.integers(n, size=m)
    say(f"bl_logprobs_backward m={m} n={n} bf16={is_bf16}")
    xd, td = device(x, is_bf16), torch.from_numpy(target.astype(np.int32)).to(DEV)
    scale = float(np.float32(0.7))
    _, lse, entropy, _, _ = bl.bl_logprobs(xd, td, scale=scale)
    g, gh, gz = rng.standard_normal((3, m)).astype(np.float32)
    for use in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        parts = [v if u else None for u, v in zip(use, (g, gh, gz))]
        want, bound = _answers.logprobs_gradient(x, target, *parts, scale=scale, bf16=is_bf16)
        on = [None if v is None else f32(v) for v in parts]
        dx = bl.bl_logprobs_backward(xd, td if use[0] else None, lse, entropy if use[1] else None, *on, scale=scale)
        near(f64(dx), want, bound)
    inside = xd.clone()
    assert bl.bl_logprobs_backward(inside, td, lse, entropy, *on, scale=scale, dlogits=inside) is inside
    assert torch.equal(inside, dx)


def test_past_two_to_the_32():
    """Rows whose elements lie past 2^32 of them."""
    m, n = 34000, 128256
    say("bl_logprobs past 2^32 elements")
    x = torch.zeros((m, n), dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(9)
    last = rows(rng, 3, n, True)
    x[-3:] = bf16(_block.bits(last))
    target = torch.full((m,), 11, dtype=torch.int32, device=DEV)
    logprob, lse, entropy, _, _ = bl.bl_logprobs(x, target)
    want = _answers.logprobs(last, np.full(3, 11))
    near(f64(lse[-3:]), want["lse"], want["lse_bound"])
    near(f64(logprob[-3:]), want["logprob"], _answers.logprob_bound(want["logprob"][:, None], want["sum_bound"])[:, 0])
    even = _answers.logprobs(np.zeros((1, n)), None)
    near(f64(entropy[:-3]), np.repeat(even["entropy"], m - 3), even["entropy_bound"])
    g = torch.zeros(m, device=DEV)
    g[-3:] = 1.0
    dx = bl.bl_logprobs_backward(x, target, lse, entropy, g, dlogits=x)
    grad, bound = _answers.logprobs_gradient(last, np.full(3, 11), np.ones(3), bf16=True)
    near(f64(dx[-3:]), grad, bound)
    assert not dx[:-3].any()


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(12)
    x = [device(rows(rng, 4, 40001, True), True) for _ in range(3)]
    target = torch.tensor([1, 2, 3, -1], dtype=torch.int32, device=DEV)
    g = f32(rng.standard_normal(4))
    say("bl_logprobs captured")

    def step(x, ws):
        out = bl.bl_logprobs(x, target, top=12, workspace=ws)
        return [*out, bl.bl_logprobs_backward(x, target, out[1], out[2], g, g)]

    ws = [torch.empty(bl.bl_logprobs_workspace_bytes(4, 40001, torch.bfloat16, 12), dtype=torch.uint8, device=DEV) for _ in range(2)]
    want = [[t.clone() for t in step(v, ws[0])] for v in x]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other = step(x[1], ws[1])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want[1]))
    held = x[0].clone()
    graphs = []
    for _ in range(2):  # two graphs over one workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(held, ws[1])
        graphs.append((graph, out))
    for i in (1, 2, 0, 1):
        held.copy_(x[i])
        graphs[i % 2][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphs[i % 2][1], want[i]))
        step(x[2], ws[0])


def test_empty_batch():
    out = bl.bl_logprobs(torch.empty((0, 50), dtype=torch.bfloat16, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), top=3)
    assert [tuple(t.shape) for t in out] == [(0,), (0,), (0,), (0, 3), (0, 3)]
