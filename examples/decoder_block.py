#!/usr/bin/env python3
"""A small decoder of BitLinear blocks with random weights: prompts through the
8-bit cache, then single tokens from a captured HIP graph.

Each block is norm -> qkv BitLinear -> rotary positions and cache -> attention
-> norm -> output BitLinear -> norm -> gate+up BitLinear with squared ReLU ->
norm -> down BitLinear, the norms before the second and the last product being
the sub-layer norms of the 2B4T block (onilabs.co, "A Two-Billion Ternary
Bet").  Every norm hands int8 rows straight to the next product; the residual
stream stays in bf16 and is added inside the norms.

  python examples/decoder_block.py [--layers 4] [--prompt 700] [--steps 64]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ternary_weight_absmean_amd as bl  # noqa: E402

EPS = 1e-5


class Block:
    """One block's weights; sizes as in the 2B-shaped stack by default."""

    def __init__(self, g: torch.Generator, hidden=2560, q_heads=20, kv_heads=5, ffn=6912):
        dev = g.device
        self.q_heads, self.kv_heads, self.dim, self.ffn = q_heads, kv_heads, hidden // q_heads, ffn
        self.n_qkv = (q_heads + 2 * kv_heads) * self.dim

        def weight(n, k):
            return torch.randn((n, k), generator=g, device=dev) * 0.02

        self.qkv = bl.bl_ternarize_pack(weight(self.n_qkv, hidden))
        self.out = bl.bl_ternarize_pack(weight(hidden, hidden))
        self.gate_up = bl.bl_ternarize_pack_glu(weight(2 * ffn, hidden))
        self.down = bl.bl_ternarize_pack(weight(hidden, ffn))
        self.norms = [1.0 + 0.1 * torch.randn(n, generator=g, device=dev) for n in (hidden, hidden, hidden, ffn)]
        self.hidden = hidden

    def forward(self, x, residual, cache, batch, rope):
        """(block output before its residual's addition, residual stream) of bf16 rows ``x`` and ``residual``
        (None for the first block): the next norm adds the two."""
        m = x.shape[0]
        xq, alpha, r, _, _ = bl.bl_rmsnorm_quant(x, self.norms[0], EPS, residual=residual)
        r = x if r is None else r
        _, qkv = bl.bl_linear(*self.qkv, xq, alpha, self.n_qkv, acc=False)
        q, k, v = qkv.view(m, -1, self.dim).split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        q = bl.bl_kv_append(cache, batch, k, v, rope=rope, q=q)
        o = bl.bl_attention(cache, batch, q).view(m, self.hidden)
        xq, alpha, *_ = bl.bl_rmsnorm_quant(o, self.norms[1], EPS)
        _, y = bl.bl_linear(*self.out, xq, alpha, self.hidden, acc=False)
        xq, alpha, r, _, _ = bl.bl_rmsnorm_quant(y, self.norms[2], EPS, residual=r)
        h = bl.bl_linear_glu(*self.gate_up, xq, alpha, self.ffn)
        xq, alpha, *_ = bl.bl_rmsnorm_quant(h, self.norms[3], EPS)
        _, y = bl.bl_linear(*self.down, xq, alpha, self.hidden, acc=False)
        return y, r


class Decoder:
    """Blocks, their caches (one per block, the same pages in each) and the page table of a fixed set of sequences."""

    def __init__(self, layers, seqs, max_tokens, device, page_tokens=64, seed=0, **block):
        g = torch.Generator(device=device).manual_seed(seed)
        self.blocks = [Block(g, **block) for _ in range(layers)]
        b = self.blocks[0]
        stride = -(-max_tokens // page_tokens)
        self.caches = [bl.KVCache.empty(seqs * stride, b.kv_heads, page_tokens, b.dim, device) for _ in range(layers)]
        # pages handed out in turn, as they would be while sequences grow together
        self.table = torch.arange(seqs * stride, dtype=torch.int32, device=device).view(stride, seqs).t().contiguous()
        self.rope = bl.Rope(bl.bl_rope_frequencies(b.dim, base=500000.0).to(device))
        self.final = 1.0 + 0.1 * torch.randn(b.hidden, generator=g, device=device)
        self.seqs, self.device, self.max_tokens = seqs, device, max_tokens

    def batch(self, start, lengths):
        """The step that gives every sequence ``lengths[s]`` tokens after its ``start[s]``."""
        offsets = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
        t = lambda v: torch.tensor(v, dtype=torch.int32, device=self.device)  # noqa: E731
        return bl.KVBatch(self.table, t(start), t(offsets), offsets[-1], max(lengths),
                          max(a + n for a, n in zip(start, lengths)))

    def forward(self, x, batch):
        """Final-norm rows (bf16) of the step's input rows (bf16)."""
        residual = None
        for block, cache in zip(self.blocks, self.caches):
            x, residual = block.forward(x, residual, cache, batch, self.rope)
        return bl.bl_rmsnorm_quant(x, self.final, EPS, residual=residual, r=False, y=True, xq=False)[3]

    def capture(self, x, start):
        """(graph, output): one token of every sequence from the rows in ``x`` at the positions in the int32 tensor
        ``start``, which each replay moves on by one."""
        offsets = torch.arange(self.seqs + 1, dtype=torch.int32, device=self.device)
        batch = bl.KVBatch(self.table, start, offsets, self.seqs, 1, self.max_tokens)
        keep = start.clone()
        side = torch.cuda.Stream()  # warm up outside the capture; the same tokens written again change nothing
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward(x, batch)
        torch.cuda.current_stream().wait_stream(side)
        start.copy_(keep)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = self.forward(x, batch)
            start.add_(1)
        self.captured = (x, batch)  # the graph reads these tensors: they stay as long as it does
        return graph, out


def norm_linear_backward(dy, r, norm_weight, packed, gamma, xq, alpha, dr=None):
    """Training: gradients of norm -> BitLinear (straight through both quantizers) for the output gradient ``dy``
    (bf16 [m][n]): (dx bf16 of the norm's input, dw of the norm, dW of the shadow weights).  ``r`` is the norm's
    input as stored, ``dr`` the gradient that reaches it past the norm."""
    n, k = dy.shape[1], r.shape[1]
    dn = bl.bl_bitlinear_backward_x(bl.bl_pack_transposed(packed, n, k), gamma, dy, k)
    dx, dw = bl.bl_rmsnorm_backward(dn, r, norm_weight, EPS, dr=dr)
    return dx, dw, bl.bl_bitlinear_backward_w(dy, xq, alpha)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=700, help="tokens of the longest of the four prompts")
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    dev = torch.device("cuda", 0)
    lengths = [max(1, a.prompt * (4 - s) // 4) for s in range(4)]
    d = Decoder(a.layers, len(lengths), a.prompt + a.steps + 1, dev)
    g = torch.Generator(device=dev).manual_seed(1)
    prompt = torch.randn((sum(lengths), d.blocks[0].hidden), generator=g, device=dev).to(torch.bfloat16)
    batch = d.batch([0] * len(lengths), lengths)
    d.forward(prompt, batch)
    torch.cuda.synchronize()
    t = time.perf_counter()
    out = d.forward(prompt, batch)
    torch.cuda.synchronize()
    took = time.perf_counter() - t
    print(f"prompts of {lengths} tokens, {a.layers} blocks: {took * 1e3:.2f} ms")
    x = out[torch.tensor([sum(lengths[:s + 1]) - 1 for s in range(len(lengths))], device=dev)].contiguous()
    start = torch.tensor(lengths, dtype=torch.int32, device=dev)
    graph, row = d.capture(x, start)
    graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps - 1):
        x.copy_(row)  # no vocabulary here: a step's output row is the next step's input
        graph.replay()
    torch.cuda.synchronize()
    took = (time.perf_counter() - t) / max(1, a.steps - 1)
    print(f"{a.steps} steps of {len(lengths)} sequences: {took * 1e6:.1f} us per step, "
          f"{took / a.layers * 1e6:.1f} us per block")
    assert torch.isfinite(row.float()).all()


if __name__ == "__main__":
    main()
