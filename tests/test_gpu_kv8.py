"""Attention over the 8-bit cache against the definition in 64 bits, over the values
that the cache stands for; bounds in kv8_util.attention_bounds."""
import math

import pytest
import torch

import kv8_util as U
from gpu_util import announce, device
from kv4_util import attention64
from test_gpu_kv8_store import DT, I32, draw, starts_of, tables
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu


class Case:
    """A cache with sequences in it, queries, and what the attention has to be."""

    def __init__(self, hq, h, d, page, dtype, q_lens, kv_lens, seed=0, k=None, v=None, q=None, width=None):
        self.hq, self.h, self.d, self.page, self.dt = hq, h, d, page, DT[dtype]
        self.dtype, self.q_lens, self.kv_lens = dtype, q_lens, kv_lens
        self.table, self.n_pages = tables(kv_lens, page, seed=seed, width=width)
        n = sum(kv_lens)
        self.k = (draw(n, h, d, dtype, seed + 1) if k is None else k).to(self.dt)
        self.v = (draw(n, h, d, dtype, seed + 2) if v is None else v).to(self.dt)
        g = torch.Generator().manual_seed(seed + 3)
        self.q = (torch.randn(sum(q_lens), hq, d, generator=g) if q is None else q).to(self.dt)
        # what a page that was never written holds: NaN scales and the largest codes
        self.cache = B.gq_kv8_empty(self.n_pages, h, d, page, device=device()).fill_(0xFF)
        if n:
            B.gq_kv8_append(self.k.to(device()), self.v.to(device()), self.cache, self.table.to(device()), I32(kv_lens),
                            starts_of(kv_lens))
        self.dq, self.dtable, self.dlens = self.q.to(device()), self.table.to(device()), I32(kv_lens)
        self.starts = None if all(n == 1 for n in q_lens) else starts_of(q_lens)

    def run(self, **kw):
        a = dict(q_starts=self.starts, max_q_len=max(self.q_lens + [0]),
                 max_kv_len=max(self.kv_lens + [0]), return_lse=True)
        a.update(kw)
        return B.gq_kv8_attention(self.dq, self.cache, self.dtable, self.dlens, **a)

    def check(self, causal=True, window=0, scale=None, dead=None, **kw):
        out, lse = self.run(causal=causal, window=window, scale=scale, **kw)
        torch.cuda.synchronize()
        out, lse = out.cpu().double(), lse.cpu().double()
        sc = self.d ** -0.5 if scale is None else scale
        r = self.hq // self.h
        most = kw.get("max_q_len", max(self.q_lens))
        at = qa = 0
        for b, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            k, sk = U.cached(self.k[at:at + kv])
            v, sv = U.cached(self.v[at:at + kv])
            q = self.q[qa:qa + n].double()
            o, l, p = attention64(q, k, v, n, kv, causal, window, sc, None if dead is None else dead[b])
            rest = self.dtype == "f16" and most * r <= 16 and n * r <= 8
            tol, ltol = U.attention_bounds(q, k, v, sk, sv, o, l, p, sc, self.dt, rest)
            e = (out[qa:qa + n] - o).abs()
            assert bool((e <= tol).all()), f"sequence {b}: off by {float((e / tol).max()):.2f} of the bound"
            none = l == -math.inf
            assert torch.equal(lse[qa:qa + n] == -math.inf, none)
            assert bool((out[qa:qa + n][none] == 0).all())
            le = (lse[qa:qa + n] - l).abs().masked_fill(none, 0.0)
            assert bool((le <= ltol).all()), f"sequence {b}: lse off by {float((le / ltol).max()):.2f} of the bound"
            at, qa = at + kv, qa + n
        return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,h,d,page,kv_lens", [
    (4, 4, 64, 16, [1, 16, 17, 300]), (6, 2, 96, 32, [31, 33, 0, 515]), (32, 8, 128, 64, [201]),
    (8, 1, 128, 16, [1000, 2, 129]), (7, 1, 256, 64, [63, 64, 65, 400]), (64, 1, 64, 16, [77, 190]),
    (20, 1, 256, 128, [600, 31]), (34, 2, 128, 16, [1300, 5]), (2, 1, 96, 1024, [1025])])
def test_single_tokens(dtype, hq, h, d, page, kv_lens):
    announce(f"kv8 decode {dtype} {hq}/{h}x{d} page {page} {kv_lens}")
    c = Case(hq, h, d, page, dtype, [1] * len(kv_lens), kv_lens)
    c.check()
    c.check(window=40)
    c.check(max_kv_len=1)                    # one workgroup per row tile
    c.check(max_kv_len=1 << 20)              # split


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,h,d,page,q_lens,kv_lens", [
    (8, 2, 128, 16, [4, 1, 3, 2], [4, 100, 35, 700]), (4, 4, 64, 32, [5, 6, 1], [5, 900, 17]),
    (8, 1, 96, 16, [4, 2], [300, 40]), (4, 2, 256, 64, [7, 16], [16, 500]),
    (4, 1, 128, 16, [65, 1, 30], [65, 400, 100]), (8, 2, 64, 16, [130, 64, 0, 3], [130, 300, 50, 3]),
    (3, 1, 96, 32, [200, 33], [457, 33]), (5, 1, 256, 64, [70, 129], [290, 129]), (64, 1, 128, 16, [9], [130]),
    (6, 2, 128, 128, [257], [1025])])
def test_several_queries(dtype, hq, h, d, page, q_lens, kv_lens):
    announce(f"kv8 prompt {dtype} {hq}/{h}x{d} page {page} {q_lens} {kv_lens}")
    c = Case(hq, h, d, page, dtype, q_lens, kv_lens, seed=5)
    c.check()
    c.check(window=33)
    c.check(causal=False)
    c.check(max_q_len=1, max_kv_len=16)      # bounds that are too small choose other kernels only
    c.check(max_q_len=sum(q_lens) + 300)


def test_queries_before_the_keys():
    """More queries than keys: the first ones stand at negative positions and see nothing."""
    for q_lens, kv in (([9], [4]), ([70], [40]), ([3, 2], [0, 1])):
        Case(4, 2, 128, 16, "bf16", q_lens, kv, seed=1).check()


@pytest.mark.parametrize("q_len", [1, 20])
def test_pages_that_do_not_exist(q_len):
    kv = 200
    c = Case(4, 1, 128, 16, "bf16", [q_len, q_len], [kv, kv], seed=2)
    dead = [torch.zeros(kv, dtype=torch.bool), torch.zeros(kv, dtype=torch.bool)]
    for b, j, number in ((0, 0, -1), (0, 5, c.n_pages), (0, 6, 2147483647), (0, 12, -7)):
        c.table[b, j] = number
        dead[b][16 * j:16 * j + 16] = True
    c.table[1] = -1
    dead[1][:] = True
    c.dtable = c.table.to(device())
    c.check(dead=dead)
    c.check(dead=dead, max_kv_len=1 << 20)
    # a query that is not finite: NaN where it sees keys, zeros where it sees none
    c.dq[0, 0, 3] = float("nan")
    c.dq[q_len, 0, 3] = float("inf")
    out, _ = c.run()
    assert bool(torch.isnan(out[0, 0]).all()) and bool((out[q_len] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("d", [64, 256])
def test_ranges(dtype, q_len, d):
    """Scales far apart from block to block, blocks of zeros, tiny and large values and
    queries, a heavy key beside thousands of light ones."""
    kv, h = 300, 2
    g = torch.Generator().manual_seed(7)
    size = lambda lo, hi: 2.0 ** (lo + (hi - lo) * torch.rand(kv // 16 + 1, 1, 1, generator=g).repeat_interleave(16, 0)[:kv])
    base = torch.randn(kv, h, d, generator=g)
    small = -20 if dtype == "f16" else -60
    zero = base * 0
    some = base.clone()
    some[32:96] = 0
    top = 10 if dtype == "f16" else 60
    for k, v, q in ((base * size(-12, 2), base * size(small, 3), 1.0), (base, some, 1.0), (some, zero, 1.0),
                    (base, base * 2.0 ** small, 1.0), (base, base * 2.0 ** top, 1.0),
                    (base * 2.0 ** -8, base, 2.0 ** 7), (base * 2.0 ** 7, base, 2.0 ** -8)):
        qq = torch.randn(q_len, 4 * h, d, generator=g) * q
        Case(4 * h, h, d, 16, dtype, [q_len], [kv], k=k, v=v, q=qq).check()
    # one query far larger in one channel than in the others
    qq = torch.randn(q_len, 4 * h, d, generator=g) * 2.0 ** -6
    qq[..., 5] = 16.0
    Case(4 * h, h, d, 16, dtype, [q_len], [kv], k=base, v=base, q=qq).check()


@pytest.mark.parametrize("q_len", [1, 20])
def test_light_weights_beside_a_heavy_one(q_len):
    """4096 keys 11 nats behind the first: together they weigh 7 % of it, and fp16 without
    room above the largest weight would lose bits of each."""
    kv, d = 4097, 64
    k = torch.zeros(kv, 1, d)
    k[:, 0, 0] = -5.0
    k[0, 0, 0] = 6.0
    v = torch.zeros(kv, 1, d)
    v[1:, 0] = 1.0
    v[0, 0] = -0.03125
    q = torch.zeros(q_len, 2, d)
    q[..., 0] = 8.0
    for dtype in ("bf16", "f16"):
        Case(2, 1, d, 16, dtype, [q_len], [kv], k=k, v=v, q=q).check(causal=False)


@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("at", [2.0 ** -30, 2.0 ** 100, 2.0 ** 120])
def test_light_weights_of_large_and_small_values(q_len, at):
    """Sums of weights far apart stay right where the values' scale is at an end of its range:
    64 keys 13 nats behind the first, which lies in a block of zeros and weighs nothing else."""
    kv, d = 1040, 64
    k = torch.zeros(kv, 1, d)
    k[:, 0, 0] = -6.5
    k[0, 0, 0] = 6.5
    v = torch.full((kv, 1, d), at)
    v[:16] = 0
    q = torch.zeros(q_len, 2, d)
    q[..., 0] = 8.0
    Case(2, 1, d, 16, "bf16", [q_len], [kv], k=k, v=v, q=q).check(causal=False)
    v[:16] = at * 2
    Case(2, 1, d, 16, "bf16", [q_len], [kv], k=k, v=v, q=q).check(causal=False)


@pytest.mark.parametrize("q_len", [1, 20])
def test_keys_of_the_largest_scale_beside_zeros(q_len):
    """A block whose scale times the query's is beyond fp32 beside keys of zeros: scores 0."""
    kv, d = 64, 64
    k = torch.zeros(kv, 1, d)
    k[16, 0, 1] = 2.0 ** 126                     # a channel in which the queries are 0
    v = torch.randn(kv, 1, d, generator=torch.Generator().manual_seed(0))
    q = torch.zeros(q_len, 2, d)
    q[..., 0] = 2.0 ** 100
    c = Case(2, 1, d, 16, "bf16", [q_len], [kv], k=k, v=v, q=q)
    out, lse = c.run(causal=False)
    mean = U.cached(c.v)[0].mean(0)
    assert bool(((out.cpu().double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -10).all())
    assert bool(((lse.cpu().double() - math.log(kv)).abs() <= 2.0 ** -18).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_sequences(dtype):
    """More sequences than lanes, empty ones among them; with and without the split, single
    tokens and prompts."""
    kv = [(i * 37) % 90 for i in range(130)] + [400]
    Case(4, 2, 64, 16, dtype, [1] * 131, kv, seed=11).check()
    c = Case(4, 2, 64, 16, dtype, [1] * 131, kv, seed=12)
    c.check(max_kv_len=1 << 20)
    q = [min(n, (i * 5) % 23) for i, n in enumerate(kv)]
    Case(4, 2, 64, 16, dtype, q, kv, seed=13).check()
    Case(6, 2, 128, 32, dtype, q, kv, seed=14).check(window=30)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,h,d,q_len,batch,bound", [
    (8, 4, 64, 1, 150, 2048), (8, 4, 64, 9, 150, 2048), (8, 2, 128, 1, 3, 1 << 20), (4, 1, 96, 5, 3, 1 << 20), (4, 1, 256, 5, 3, 1 << 20)])
def test_bounds_that_promise_much(dtype, hq, h, d, q_len, batch, bound):
    """Where the bounds say that more is read than the caches hold, codes pass them by."""
    kv = [q_len + (i * 29) % 130 for i in range(batch)]
    Case(hq, h, d, 16, dtype, [q_len] * batch, kv, seed=15).check(max_kv_len=bound)


def test_cache_of_more_than_4_gib():
    """Pages beyond 2^32 bytes: appended, read back and attended to."""
    d, page, n_pages = 256, 1024, 8300
    cache = B.gq_kv8_empty(n_pages, 1, d, page, device=device())
    assert cache.numel() > 1 << 32
    table = torch.tensor([[8299, 5], [8200, 8298]], dtype=torch.int32)
    k, v = draw(1100 + 1500, 1, d, "bf16", 1), draw(2600, 1, d, "bf16", 2)
    lens = [1100, 1500]
    dt = table.to(device())
    B.gq_kv8_append(k.to(device()), v.to(device()), cache, dt, I32(lens), starts_of(lens))
    slot = torch.tensor([8299 * 1024 + 7, 8298 * 1024 + 475], device=device())
    got = B.gq_kv8_read(cache, slot, d, torch.float32)[1].cpu()
    want = [U.cached(v[:1100])[0], U.cached(v[1100:])[0]]
    assert torch.equal(got, torch.stack((want[0][7], want[1][1499])).float())
    q = torch.randn(2 + 40, 4, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    for n in (1, 20):
        out = B.gq_kv8_attention(q[:2 * n].to(device()), cache, dt, I32(lens), I32([0, n, 2 * n]), n, 1500).cpu().double()
        at = 0
        for b, m in enumerate(lens):
            kk, sk = U.cached(k[at:at + m])
            vv, sv = U.cached(v[at:at + m])
            qq = q[b * n:b * n + n].double()
            o, l, p = attention64(qq, kk, vv, n, m, True, 0, d ** -0.5)
            tol, _ = U.attention_bounds(qq, kk, vv, sk, sv, o, l, p, d ** -0.5, torch.bfloat16, False)
            assert bool(((out[b * n:b * n + n] - o).abs() <= tol).all())
            at += m


def test_views_rows_left_alone_and_scale():
    c = Case(8, 2, 128, 16, "bf16", [3, 2], [50, 20], seed=3)
    want, wl = c.run()
    qkv = torch.zeros(9, 12, 128, dtype=torch.bfloat16, device=device())
    qkv[:5, 1:9] = c.dq
    out = torch.full((9, 8, 128), 5.0, dtype=torch.bfloat16, device=device())
    lse = torch.full((9, 8), 5.0, device=device())
    B.gq_kv8_attention(qkv[:, 1:9], c.cache, c.dtable, c.dlens, I32([0, 3, 5]), 3, 50, out=out, lse=lse)
    assert torch.equal(out[:5], want) and torch.equal(lse[:5], wl)
    assert bool((out[5:] == 5).all()) and bool((lse[5:] == 5).all())
    c.check(scale=0.31)
    c.check(scale=2.0)


def test_head_tables():
    """Pages of each head's own: one call against one per head."""
    h, d, page, nb = 4, 128, 16, 3
    c = Case(8, h, d, page, "f16", [1] * nb, [400, 90, 33], seed=4)
    g = torch.Generator().manual_seed(0)
    tab = torch.full((nb, h, 7), -1, dtype=torch.int32)
    for b, n in enumerate((25, 6, 3)):
        for x in range(h):
            take = torch.randperm(n, generator=g)[:min(7, n - 1)].sort().values
            tab[b, x, :take.numel()] = c.table[b, take]
    lens = I32([7 * 16 - 3, 5 * 16 - 1, 17])
    for most in (1, 1 << 20):
        out, lse = B.gq_kv8_attention(c.dq, c.cache, tab.to(device()), lens, max_kv_len=most, return_lse=True)
        for x in range(h):
            o1, l1 = B.gq_kv8_attention(c.dq, c.cache, tab[:, x].contiguous().to(device()), lens, max_kv_len=most, return_lse=True)
            assert torch.equal(out[:, 2 * x:2 * x + 2], o1[:, 2 * x:2 * x + 2])
            assert torch.equal(lse[:, 2 * x:2 * x + 2], l1[:, 2 * x:2 * x + 2])
    # a prompt's kernel reads them too
    same = c.table[:1, None, :25].repeat(1, h, 1).contiguous().to(device())
    q = torch.randn(60, 8, d, generator=g).half().to(device())
    a = B.gq_kv8_attention(q, c.cache, same, I32([400]), I32([0, 60]), 60, 400)
    b = B.gq_kv8_attention(q, c.cache, c.dtable[:1], I32([400]), I32([0, 60]), 60, 400)
    assert torch.equal(a, b)


def test_empty_calls_and_lengths_out_of_range():
    c = Case(4, 2, 64, 16, "bf16", [1, 1], [40, 20], seed=6)
    assert B.gq_kv8_attention(c.dq[:0], c.cache, c.dtable[:0], c.dlens[:0]).shape == (0, 4, 64)
    out, lse = B.gq_kv8_attention(c.dq, c.cache, c.dtable, I32([-5, 0]), return_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())
    out, lse = B.gq_kv8_attention(c.dq, c.cache, c.dtable[:, :0].contiguous(), c.dlens, return_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())
    cap = c.dtable.shape[1] * 16                         # lengths past the table count as its end
    a = B.gq_kv8_attention(c.dq[:1], c.cache, c.dtable[:1], I32([cap + 1000]))
    assert torch.equal(a, B.gq_kv8_attention(c.dq[:1], c.cache, c.dtable[:1], I32([cap])))


@pytest.mark.parametrize("q_len,kv", [(1, 3000), (1, 100), (40, 300)])
def test_same_result_every_time_streams_and_graphs(q_len, kv):
    c = Case(8, 2, 128, 64, "bf16", [q_len] * 3, [kv, kv - 70, q_len], seed=8)
    want, wl = c.run()
    for _ in range(3):
        a, b = c.run()
        assert torch.equal(a, want) and torch.equal(b, wl)
    # two streams at once, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        outs.append(c.run(stream=s))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, wl)
    # a raw stream handle needs the caller's workspace where one is used
    args = dict(q_starts=c.starts, max_q_len=q_len, max_kv_len=kv)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=device())
    raw = torch.cuda.current_stream().cuda_stream
    assert torch.equal(B.gq_kv8_attention(c.dq, c.cache, c.dtable, c.dlens, stream=raw, workspace=ws, **args), want)
    # two graphs replayed in turn with eager work between
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = c.run(**args)
        graphs.append((g, o))
    q0 = c.dq.clone()
    for i in range(4):
        c.dq.copy_(q0 * (1 + i))
        eager = c.run()
        for g, o in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], eager[0]) and torch.equal(o[1], eager[1])


def test_long_context_split():
    c = Case(8, 1, 128, 64, "f16", [1, 1], [20001, 3], seed=9)
    c.check()
    c = Case(4, 1, 64, 16, "bf16", [2, 2], [12000, 5000], seed=10)
    c.check()
