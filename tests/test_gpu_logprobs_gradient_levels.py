"""GPU checks of the gradient of log probabilities for rows far from 0: it does not
change with a row's level, so neither does its bound.

A weight's relative error in the gradient is the sum's (as _answers derives it for
the forward call; the gradient's own sums are no longer), the exponent's roundings,
relative to log p and log S, and one rounding of lse while |lse| is below the level
from which on the sum is taken again (64 for fp32, 512 for bf16)."""
import numpy as np
import pytest
import torch

import _answers
import _block
import ternary_weight_absmean_amd as bl
from _block import U16, U32
from _gpu import DEV, f32, say
from test_gpu_logprobs import check, device, f64, near, rows
from test_gpu_logprobs_levels import LEVELS

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)


def gradient(x, target, g, gh, gz, scale, bf16):
    """(gradient, bound of its error) in 64 bits."""
    m, n = x.shape
    x = np.asarray(x, np.float64)
    want, _ = _answers.logprobs_gradient(x, target, g, gh, gz, scale, bf16)
    r = _answers.logprobs(x, None, scale)
    level = np.abs(r["lse"])
    level = np.where(level < (512 if bf16 else 64), level, 0.0)
    log_s = np.abs(r["lse"] - x.max(axis=1) * scale)  # at most log n; lost in 64 bits it is small against sum_bound
    log_p = np.where(r["p"] > 0, r["log_p"], 0.0)
    off = (r["sum_bound"] + U32 * (3 * level + 8 * np.minimum(log_s, np.log(n)) + 64))[:, None] + U32 * 8 * np.abs(log_p)
    g, gh, gz = (np.zeros(m) if v is None else np.asarray(v, np.float64) for v in (g, gh, gz))
    known = (np.asarray(target) >= 0) & (np.asarray(target) < n)
    g = np.where(known, g, 0.0)[:, None]
    gh, gz = gh[:, None], gz[:, None]
    size = np.abs(g) + np.abs(gz) + np.abs(gh) * (np.abs(log_p) + r["entropy"][:, None])
    bound = scale * r["p"] * (size * (off + 8 * U32) + np.abs(gh) * (r["entropy_bound"][:, None] + off))
    hit = np.zeros((m, n))
    hit[np.arange(m)[known], np.asarray(target)[known]] = 1.0
    # p is held in fp32: one below 2^-126 may be 0, which takes at most 2^-126 off p, times what p is multiplied by
    bound = bound + 4 * U32 * scale * np.abs(g) * hit + 2.0 ** -126 * scale * size
    return want, bound + (U16 if bf16 else U32) * (np.abs(want) + bound) + 2.0 ** -120


def check_gradient(x, xd, target, lse, entropy, parts, scale, is_bf16, **kw):
    g, gh, gz = parts
    want, bound = gradient(x, target, g, gh, gz, scale, is_bf16)
    td = torch.from_numpy(np.asarray(target, np.int32)).to(DEV)
    on = [None if v is None else f32(v) for v in parts]
    dx = bl.bl_logprobs_backward(xd, td, lse, entropy, *on, scale=scale, **kw)
    near(f64(dx), want, bound)
    return dx, bound


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("n,lead", [(1, 0), (7, 1), (300, 0), (5003, 3), (70001, 0), (128256, 5)])
def test_gradients_at_any_level(n, lead, is_bf16):
    rng = np.random.default_rng(n + lead)
    x = rows(rng, len(LEVELS), n, False) + np.asarray(LEVELS, np.float32)[:, None]
    x = _block.bf16_round(x) if is_bf16 else x
    target = rng.integers(n, size=len(LEVELS))
    target[3] = -1
    say(f"bl_logprobs levels n={n} lead={lead} bf16={is_bf16}")
    xd = device(x, is_bf16, lead, 2)
    scale = float(np.float32(0.7))
    _, lse, entropy, _, _ = check(x, xd, target, scale, min(n, 4))
    g, gh, gz = rng.standard_normal((3, len(LEVELS))).astype(np.float32)
    for parts in ((g, None, None), (g, gh, gz)):
        dx, bound = check_gradient(x, xd, target, lse, entropy, parts, scale, is_bf16)
        if parts[1] is None:  # weights of a row sum to 1, so the gradient of one token's score sums to 0
            total = np.where(target >= 0, f64(dx).sum(axis=1), 0.0)
            assert (np.abs(total) <= bound.sum(axis=1)).all()
    whole = torch.full((len(LEVELS), lead + n + 3), 5.0, dtype=xd.dtype, device=DEV)
    check_gradient(x, xd, target, lse, entropy, parts, scale, is_bf16, dlogits=whole[:, lead:lead + n])  # begins as rows of x do or not
    assert (whole[:, :lead] == 5.0).all() and (whole[:, lead + n:] == 5.0).all()
    again, _ = check_gradient(x, xd.clone(), target, lse, entropy, parts, scale, is_bf16)
    here = xd.clone()
    assert bl.bl_logprobs_backward(here, torch.from_numpy(target.astype(np.int32)).to(DEV), lse, entropy, *[f32(v) for v in parts],
                                   scale=scale, dlogits=here) is here
    assert torch.equal(here, again)


@pytest.mark.parametrize("is_bf16", [True, False])
@pytest.mark.parametrize("n", [2, 60, 3000, 70000])
def test_gradients_of_rows_of_the_lowest_value(n, is_bf16):
    """A row wholly masked by the type's lowest value: all alike, 1 / n each."""
    low = float(torch.finfo(torch.bfloat16).min) if is_bf16 else float(np.finfo(np.float32).min)
    x = np.full((3, n), low, np.float32)
    x[1, ::2] = -np.inf
    x[2, 0] = 5.0
    target = np.array([1, n - 1 - (n + 1) % 2, 1])
    say(f"bl_logprobs lowest n={n} bf16={is_bf16}")
    xd = device(x, is_bf16)
    _, lse, entropy, _, _ = check(x, xd, target)
    g, gh, gz = np.random.default_rng(n).standard_normal((3, 3)).astype(np.float32)
    dx, bound = check_gradient(x, xd, target, lse, entropy, (g, None, None), 1.0, is_bf16)
    assert (np.abs(f64(dx).sum(axis=1)) <= bound.sum(axis=1)).all()
    check_gradient(x, xd, target, lse, entropy, (g, gh, gz), 1.0, is_bf16)


def test_gradients_at_a_level_against_differences():
    """Differences of the forward call's own log probabilities and entropies, at logits around 300 and -300 and in steps that
    these take exactly."""
    rng = np.random.default_rng(4)
    n = 40
    say("bl_logprobs differences at a level")
    for level, step in ((300.0, 2.0 ** -9), (-300.0, 2.0 ** -9)):
        x = (np.round((rng.standard_normal((1, n)) * 2) * 512) / 512 + level).astype(np.float32)
        g, gh = 1.0, 0.5
        total = lambda x: sum(w * f64(t) for w, t in zip((g, gh), [bl.bl_logprobs(x, t)[i] for i in (0, 2)]))  # noqa: E731
        at = np.concatenate([x + s * step * np.eye(n, dtype=np.float32) for s in (1, -1)])
        assert np.array_equal(at.astype(np.float64), np.concatenate([x.astype(np.float64) + s * step * np.eye(n) for s in (1, -1)]))
        t = torch.full((2 * n,), 7, dtype=torch.int32, device=DEV)
        value = total(device(at, False))
        diff = (value[:n] - value[n:]) / (2 * step)
        xd = device(x, False)
        one = t[:1].contiguous()
        _, lse, entropy, _, _ = bl.bl_logprobs(xd, one)
        dx = f64(bl.bl_logprobs_backward(xd, one, lse, entropy, f32([g]), f32([gh])))[0]
        # each value is off by its bound (log probabilities and entropies are below 12 here), the difference by a third
        # derivative (at most 10 for |log p| below 12) times step^2 / 6
        r = _answers.logprobs(at, np.full(2 * n, 7))
        off = _answers.logprob_bound(r["logprob"][:, None], r["sum_bound"])[:, 0] + gh * r["entropy_bound"]
        _, bound = gradient(x, [7], [g], [gh], None, 1.0, False)
        assert (np.abs(dx - diff) <= (off[:n] + off[n:]) / (2 * step) + 10 * step ** 2 / 6 + bound[0]).all()
