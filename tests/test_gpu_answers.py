"""The operators for many answers to one prompt together, as
examples/decoder_block.py uses them: beams over shared pages against beams that
each hold a copy of all their pages, and the gradients of given tokens' scores."""
import numpy as np
import pytest
import torch

import _answers
import _block
import ternary_weight_absmean_amd as bl
from _gpu import DEV, bf16, bf16_bits_to_f64, f32, host, say
from test_gpu_decoder_example import SMALL, ex

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected only where a GPU exists
    pytest.skip("no GPU visible", allow_module_level=True)

WORDS = 1000


class Copies(ex.Beams):
    """Beams that share nothing: every page of a chosen parent is copied, by plain indexing."""

    def pages(self, parent):
        page, stride = self.pool.page_tokens, self.table.shape[1]
        base = 0 if getattr(self, "side", 1) else self.width * stride
        self.side = 0 if base else 1
        if self.caches.caches[0].pages < 2 * self.width * stride + stride:  # room for two sets, once
            more = 2 * self.width * stride + stride
            b = self.decoder.blocks[0]
            grown = []
            for old in self.caches.caches:
                new = bl.KVCache.empty(more, b.kv_heads, page, b.dim, DEV)
                for name in ("k", "v", "k_absmax", "v_absmax"):  # the prompt's pages move behind both sets
                    getattr(new, name)[2 * self.width * stride:] = getattr(old, name)[self.table[0].clamp(min=0).long()]
                grown.append(new)
            self.decoder.caches, self.caches = grown, bl.KVCaches(grown)
            self.table = torch.arange(stride, dtype=torch.int32, device=DEV)[None] + 2 * self.width * stride
        mine = torch.arange(self.width * stride, dtype=torch.int32, device=DEV).view(self.width, stride) + base
        for cache in self.caches.caches:
            for t in (cache.k, cache.v, cache.k_absmax, cache.v_absmax):
                t[mine.long()] = t[self.table[parent.long()].long()].clone()
        self.table, self.length = mine, self.length[parent.long()]
        return bl.KVBatch(self.table, self.length, self.offsets, self.width, 1, self.max_len)

    def end(self):
        pass


@pytest.mark.parametrize("prompt,width,steps,page", [(150, 5, 24, 16), (64, 3, 40, 32), (7, 4, 20, 16), (400, 12, 10, 64)])
def test_beams_with_shared_pages_equal_beams_with_copies(prompt, width, steps, page):
    """The same codes in other pages, the same kernels: every token and score is equal, bit by bit."""
    words = ex.Vocabulary(WORDS, SMALL["hidden"], DEV, seed=3)
    text = torch.randint(WORDS, (prompt,), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV, dtype=torch.int32)
    say(f"beams prompt={prompt} width={width} steps={steps} page={page}")
    both = []
    for kind in (ex.Beams, Copies):
        decoder = ex.Decoder(2, 1, prompt + steps, DEV, page_tokens=page, seed=5, **SMALL)
        beams = kind(decoder, words, text, width, steps, page_tokens=page)
        trace = []
        for _ in range(steps):
            beams.step()
            trace.append((beams.score.clone(), beams.y.clone()))
        both.append((beams, trace))
    (a, at), (b, bt) = both
    for (score, y), (other, z) in zip(at, bt):
        assert torch.equal(score, other) and torch.equal(y, z)
    assert torch.equal(a.answers, b.answers) and len({tuple(r) for r in a.answers.tolist()}) == width
    assert int(a.short) == 0
    # every beam's pages, and no others, are in use; the prompt's full ones by all beams
    held = [e for row in a.table.tolist() for e in row if e >= 0]
    refs = host(a.pool.refs)
    assert refs.sum() == len(held) and (refs[np.unique(held)] == np.unique(held, return_counts=True)[1]).all()
    assert (refs == width).sum() >= prompt // page
    a.end()
    assert not a.pool.refs.any()


def test_scores_of_given_tokens_and_their_gradients():
    rng = np.random.default_rng(6)
    m, hidden = 7, SMALL["hidden"]
    words = ex.Vocabulary(WORDS // 64 * 64, hidden, DEV, seed=7)
    y = _block.bf16_round(rng.standard_normal((m, hidden)).astype(np.float32))
    target = rng.integers(words.words, size=m)
    target[3] = -1
    g, gh = rng.standard_normal((2, m)).astype(np.float32)
    say("scores and gradients of given tokens")
    yd, td = bf16(_block.bits(y)), torch.from_numpy(target.astype(np.int32)).to(DEV)
    logits, xq, alpha = words.logits(yd)
    x = bf16_bits_to_f64(host(logits))
    logprob, entropy, dy, dw = words.score_backward(yd, td, f32(g), f32(gh))
    want = _answers.logprobs(x, target)
    bound = _answers.logprob_bound(want["logprob"][:, None], want["sum_bound"])[:, 0]
    assert (np.abs(host(logprob) - want["logprob"]) <= bound).all()
    assert (np.abs(host(entropy) - want["entropy"]) <= want["entropy_bound"]).all()
    grad, off = _answers.logprobs_gradient(x, target, g, gh, None, 1.0, bf16=True)
    # straight through the layer, as it documents: dx = gamma dy q, dW = dy^T (alpha / 127 xq)
    q = host(bl.bl_unpack_ternary(words.head[0], words.words, hidden)).astype(np.float64)
    gamma = float(host(words.head[1])[0])
    terms = gamma * (np.abs(grad) + off) @ np.abs(q)
    assert (np.abs(host(dy) - gamma * grad @ q) <= gamma * off @ np.abs(q) + terms * (words.words + 2) * _block.U32).all()
    xhat = host(xq).astype(np.float64) * host(alpha).astype(np.float64)[:, None] / 127
    terms = (np.abs(grad) + off).T @ np.abs(xhat)
    assert (np.abs(host(dw) - grad.T @ xhat) <= off.T @ np.abs(xhat) + terms * (m + 2) * _block.U32).all()
