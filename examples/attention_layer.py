"""One attention layer served in 4 bits: INT4 projections and a 4-bit key/value cache.

    python examples/attention_layer.py [--prompts 700 33 1] [--steps 8]

Several prompts of uneven length enter the cache in one call each of the qkv
projection, ``gq_kv4_write`` and ``gq_kv4_attention``; then every sequence takes
single-token steps, which are captured into a graph once and replayed.  The same
layer in float32 torch, over the values that the weights and the cache stand for,
says how far the results are off.  Weights are random; the default sizes are the
Llama-3-8B layer of the benchmark.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w4a16_dequant_gemm_group_amd import binding as B


class AttentionLayer:
    """qkv projection, rotary positions, paged 4-bit cache, attention, o projection."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, group=128, page=64, n_pages=256,
                 dtype=torch.bfloat16, seed=0):
        self.hq, self.hkv, self.d, self.g, self.page, self.dtype = q_heads, kv_heads, head_dim, group, page, dtype
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.qkv = self._weight((q_heads + 2 * kv_heads) * head_dim, hidden, gen)
        self.o = self._weight(hidden, q_heads * head_dim, gen)
        self.cache = B.gq_kv4_empty(n_pages, kv_heads, head_dim, page, group)
        self.free = list(range(n_pages))
        self.freq, _ = B.gq_rope_frequencies(head_dim, 10000.0)

    def _weight(self, n, k, gen):
        w = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(self.dtype)
        codes, scales, zeros = B.gq_quantize_groups(w, 4, self.g)
        return B.gq_pack_int4(codes), scales, zeros

    def _matmul(self, x, w):
        f16 = "_f16" if self.dtype == torch.float16 else ""
        kind = "gemv" if x.shape[0] <= 16 else "gemm"
        return getattr(B, f"gq_w4a16_{kind}{f16}")(x, *w, group_size=self.g)

    def pages_for(self, lengths, room):
        """A page table for sequences that may grow to lengths + room tokens."""
        need = [-(-(n + room) // self.page) for n in lengths]
        table = torch.zeros(len(need), max(need), dtype=torch.int32)
        for b, n in enumerate(need):
            for i in range(n):
                table[b, i] = self.free.pop()
        return table.cuda()

    def slots(self, table, seq, pos):
        return table[seq, pos // self.page].long() * self.page + pos % self.page

    def forward(self, x, pos, slots, table, kv_lens, q_starts=None, max_q_len=1, max_kv_len=None):
        """x [tokens, hidden] -> [tokens, hidden]; the tokens' keys and values enter
        the cache at `slots` and every token attends to its sequence so far."""
        t = x.shape[0]
        qkv = self._matmul(x, self.qkv).view(t, self.hq + 2 * self.hkv, self.d)
        turned = B.gq_rope(qkv[:, :self.hq + self.hkv], pos, self.freq)
        q, k = turned[:, :self.hq], turned[:, self.hq:]
        v = qkv[:, self.hq + self.hkv:]                       # a strided slice, taken as it is
        B.gq_kv4_write(k, v, self.cache, slots, self.g)
        out = B.gq_kv4_attention(q, self.cache, table, kv_lens, self.g, q_starts=q_starts, max_q_len=max_q_len,
                                 max_kv_len=max_kv_len)
        return self._matmul(out.view(t, -1), self.o), q

    def reference(self, q, table, lens, q_lens):
        """The attention and the o projection in float32 torch over the cached values."""
        wo = B.gq_dequantize(*self.o, group_size=self.g)
        outs, at = [], 0
        for b, (n, m) in enumerate(zip(lens, q_lens)):
            pos = torch.arange(n, device="cuda")
            k, v = B.gq_kv4_read(self.cache, self.slots(table, b, pos), self.d, self.g, out_dtype=torch.float32)
            r = self.hq // self.hkv
            k, v = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
            qb = q[at:at + m].float()
            out = torch.empty_like(qb)
            seen = pos <= torch.arange(n - m, n, device="cuda")[:, None]
            for h in range(self.hq):
                s = qb[:, h] @ k[:, h].T.contiguous() / math.sqrt(self.d)
                out[:, h] = torch.softmax(s.masked_fill(~seen, -math.inf), -1) @ v[:, h].contiguous()
            outs.append(out.view(m, -1) @ wo.T.contiguous())
            at += m
        return torch.cat(outs)


def run(prompts=(700, 33, 1), steps=8, **sizes):
    """Serve the prompts and `steps` tokens each; the largest relative error seen."""
    layer = AttentionLayer(**sizes)
    hidden = layer.o[0].shape[0]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rel = lambda y, ref: float((y.float() - ref).norm() / ref.norm())
    prompts = list(prompts)
    table = layer.pages_for(prompts, steps)
    most = max(prompts) + steps

    # the prompts, in one call
    x = torch.randn(sum(prompts), hidden, generator=gen, device="cuda").to(layer.dtype)
    pos = torch.cat([torch.arange(n, device="cuda") for n in prompts])
    seq = torch.cat([torch.full((n,), b, device="cuda") for b, n in enumerate(prompts)])
    starts = torch.tensor([0] + prompts).cumsum(0).int().cuda()
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    y, q = layer.forward(x, pos, layer.slots(table, seq, pos), table, lens, starts, max(prompts), max(prompts))
    worst = rel(y, layer.reference(q, table, prompts, prompts))

    # single tokens: one graph, replayed with new inputs and lengths
    nb = len(prompts)
    x1 = torch.zeros(nb, hidden, dtype=layer.dtype, device="cuda")
    p1, each = lens.long(), torch.arange(nb, device="cuda")

    def step():
        return layer.forward(x1, p1, layer.slots(table, each, p1), table, lens, max_kv_len=most)
    lens += 1
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()                                   # what is allocated once is allocated before the capture
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, q = step()
    for i in range(steps):
        x1.copy_(torch.randn(nb, hidden, generator=gen, device="cuda"))
        graph.replay()
        worst = max(worst, rel(y, layer.reference(q, table, [n + i + 1 for n in prompts], [1] * nb)))
        p1 += 1
        lens += 1
    return worst


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 33, 1])
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    print(f"largest relative error against float32 over the stored values: {run(a.prompts, a.steps):.2e}")


if __name__ == "__main__":
    main()
