"""One attention layer for long contexts: INT4 projections, rotary positions scaled beyond
the trained length, an 8-bit key/value cache, and single tokens that read only a few pages.

    python examples/sparse_layer.py [--prompts 5000 700 33] [--steps 8] [--keep 16]

The prompts enter the cache and attend to all of it; then every sequence takes single-token
steps, captured into a graph once and replayed, in which each query and key/value head
chooses `keep` pages by the bounds that the cache keeps of their keys.  The same layer in
float32 torch, over the values that the weights and the cache stand for, says how far the
results are off, and attention over all pages how much of it the chosen ones make.  Weights
are random (attention spreads over all keys then: a trained layer's is far less even); the
default sizes are the Llama-3-8B layer of the benchmark.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from attention_layer import AttentionLayer, B


class SparseLayer(AttentionLayer):
    def __init__(self, keep=16, first=1, last=2, trained=8192, stretch=8.0, **sizes):
        super().__init__(**sizes)
        self.keep, self.first, self.last = keep, first, last
        n_pages = self.cache.shape[0]
        self.cache = B.gq_kv8_empty(n_pages, self.hkv, self.d, self.page)
        self.bounds = B.gq_kv8_bounds_empty(n_pages, self.hkv, self.d, self.dtype)
        self.freq, self.amplitude = B.gq_rope_frequencies(self.d, 10000.0, "yarn", factor=stretch, original_length=trained,
                                                          low=1.0, high=32.0)

    def forward(self, x, pos, table, kv_lens, starts=None, max_q_len=1, max_kv_len=None):
        """x [tokens, hidden] -> ([tokens, hidden], queries, pages, their lengths); the tokens enter
        the cache.  With `starts` (prompts) every token attends to its sequence so far, without
        (single tokens) to the pages that its heads choose."""
        t = x.shape[0]
        qkv = self._matmul(x, self.qkv).view(t, self.hq + 2 * self.hkv, self.d)
        turned = B.gq_rope(qkv[:, :self.hq + self.hkv], pos, self.freq, amplitude=self.amplitude)
        q, k, v = turned[:, :self.hq], turned[:, self.hq:], qkv[:, self.hq + self.hkv:]
        B.gq_kv8_append(k, v, self.cache, table, kv_lens, starts, self.bounds)
        if starts is not None:
            out = B.gq_kv8_attention(q, self.cache, table, kv_lens, starts, max_q_len, max_kv_len)
            return self._matmul(out.view(t, -1), self.o), q, None, None
        pages, seen = B.gq_kv8_select(q, self.bounds, table, kv_lens, self.keep, self.page, max_kv_len=max_kv_len,
                                      first=self.first, last=self.last)
        out = B.gq_kv8_attention(q, self.cache, pages, seen)
        return self._matmul(out.view(t, -1), self.o), q, pages, seen

    def reference(self, q, table, lens, q_lens, pages=None, seen=None):
        """The attention (over `pages` where given) and the o projection in float32 torch."""
        wo = B.gq_dequantize(*self.o, group_size=self.g)
        r, outs, at = self.hq // self.hkv, [], 0
        for b, (n, m) in enumerate(zip(lens, q_lens)):
            out = torch.empty(m, self.hq, self.d, device="cuda")
            for h in range(self.hkv):
                row = table[b] if pages is None else pages[b, h]
                n_keys = n if pages is None else int(seen[b])
                p = torch.arange(n_keys, device="cuda")
                k, v = B.gq_kv8_read(self.cache, row[p // self.page].long() * self.page + p % self.page, self.d, torch.float32)
                hidden = p > torch.arange(n_keys - m, n_keys, device="cuda")[:, None]
                for y in range(h * r, (h + 1) * r):
                    s = q[at:at + m, y].float() @ k[:, h].T.contiguous() / math.sqrt(self.d)
                    out[:, y] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[:, h].contiguous()
            outs.append(out.view(m, -1) @ wo.T.contiguous())
            at += m
        return torch.cat(outs)


def run(prompts=(5000, 700, 33), steps=8, **sizes):
    """Serve the prompts and `steps` tokens each: the largest relative error seen, and the
    largest distance of a step's result from that of attention over all pages."""
    prompts = list(prompts)
    page = sizes.get("page", 64)
    sizes.setdefault("n_pages", sum(-(-(n + steps) // page) for n in prompts) + 1)
    layer = SparseLayer(**sizes)
    hidden = layer.o[0].shape[0]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rel = lambda y, ref: float((y.float() - ref).norm() / ref.norm())
    table = layer.pages_for(prompts, steps)
    most = max(prompts) + steps

    x = torch.randn(sum(prompts), hidden, generator=gen, device="cuda").to(layer.dtype)
    pos = torch.cat([torch.arange(n, device="cuda") for n in prompts])
    starts = torch.tensor([0] + prompts).cumsum(0).int().cuda()
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    y, q, _, _ = layer.forward(x, pos, table, lens, starts, max(prompts), max(prompts))
    worst, apart = rel(y, layer.reference(q, table, prompts, prompts)), 0.0

    nb = len(prompts)
    x1 = torch.randn(nb, hidden, generator=gen, device="cuda").to(layer.dtype)
    p1 = lens.long()
    lens += 1
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):              # the first step, in which what is set up once is
        layer.forward(x1, p1, table, lens, max_kv_len=most)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, q, pages, seen = layer.forward(x1, p1, table, lens, max_kv_len=most)
    for i in range(1, steps):
        x1.copy_(torch.randn(nb, hidden, generator=gen, device="cuda"))
        p1 += 1
        lens += 1
        graph.replay()
        now = [n + i + 1 for n in prompts]
        worst = max(worst, rel(y, layer.reference(q, table, now, [1] * nb, pages, seen)))
        apart = max(apart, rel(y, layer.reference(q, table, now, [1] * nb)))
    return worst, apart


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", type=int, nargs="+", default=[5000, 700, 33])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--keep", type=int, default=16)
    a = ap.parse_args()
    worst, apart = run(a.prompts, a.steps, keep=a.keep)
    print(f"largest relative error against float32 over the stored values: {worst:.2e}")
    print(f"largest distance from attention over all pages: {apart:.2e}")


if __name__ == "__main__":
    main()
