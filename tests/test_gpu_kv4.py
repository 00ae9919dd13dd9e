"""The 4-bit key/value cache on the GPU against its definition in 64 bits:
stored values exactly, attention within bounds that count the roundings."""
import math

import pytest
import torch

from gpu_util import announce
from kv4_util import attention64, attention_bounds, quantise64
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
LAYOUTS = [(128, 128, False), (128, 128, True), (128, 64, True), (128, 32, False), (64, 64, False), (64, 32, True),
           (96, 96, False), (96, 32, True), (256, 256, True), (256, 128, False), (256, 64, False), (256, 32, True)]


def rows(gen, t, h, d, dtype):
    x = torch.randn(t, h, d, generator=gen) * torch.exp(torch.randn(t, h, 1, generator=gen))
    return (x + 0.5 * torch.randn(h, d, generator=gen)).to(dtype)


def fill_random(cache, gen):
    """Every byte of an unwritten cache set: scales of any kind, NaN and infinity too."""
    cache.copy_(torch.randint(0, 256, cache.shape, generator=gen, dtype=torch.uint8))
    cache[..., ::7] = 0xFF


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g,sym", LAYOUTS)
def test_write_read_exact(d, g, sym, dtype):
    gen = torch.Generator().manual_seed(d + g + sym)
    for t, h, page, spread in ((1, 3, 16, True), (37, 2, 32, True), (150, 2, 64, False)):
        announce(f"kv4 write/read d={d} g={g} sym={sym} {dtype} t={t}")
        n_pages = t // page + 3
        k, v = rows(gen, t, h, d, DT[dtype]), rows(gen, t, h, d, DT[dtype])
        k[0, 0] = 0.0                                   # a group of zeros: scale 1
        v[0, 0, :g] = 3.5                               # no negative value: lo = 0
        v[t - 1, 0] = -v[t - 1, 0].abs()                # no positive one
        k[t - 1, 1] *= 2.0 ** -20                       # scales below fp16's normal range
        if dtype == "bf16":
            k[t // 2, 0] *= 2.0 ** 30                   # scales beyond it
        slots = torch.randperm(n_pages * page, generator=gen)[:t] if spread else torch.arange(5, 5 + t)
        cache = B.gq_kv4_empty(n_pages, h, d, page, g, sym)
        fill_random(cache, gen)
        before = cache.clone()
        B.gq_kv4_write(k.cuda(), v.cuda(), cache, slots.cuda(), g, sym)
        k32, v32 = B.gq_kv4_read(cache, slots.cuda(), d, g, sym, torch.float32)
        for got, x in ((k32, k), (v32, v)):
            want, _, _ = quantise64(x, g, sym)
            assert torch.equal(got.cpu().double(), want)
        for odt in (torch.bfloat16, torch.float16):
            ko, vo = B.gq_kv4_read(cache, slots.cuda(), d, g, sym, odt)
            assert torch.equal(ko, k32.to(odt)) and torch.equal(vo, v32.to(odt))
        # nothing else was touched: writing the old bytes' slots back is a no-op elsewhere
        row = d // 2 + (2 if sym else 4) * (d // g)
        assert int((cache != before).sum()) <= 2 * t * h * row


def test_ties_round_to_even():
    # scale exactly 2 (symmetric: 14 / 7): odd integers lie on ties
    x = torch.arange(-14, 18).float()[:32].clamp(-14, 14).to(torch.float16)
    k = x.repeat(2).reshape(1, 1, 64).clone()
    cache = B.gq_kv4_empty(1, 1, 64, 16, 32, True)
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    B.gq_kv4_write(k.cuda(), -k.cuda(), cache, slots, 32, True)
    k32, v32 = B.gq_kv4_read(cache, slots, 64, 32, True, torch.float32)
    assert torch.equal(k32.cpu().double(), quantise64(k, 32, True)[0])
    assert torch.equal(v32.cpu().double(), quantise64(-k, 32, True)[0])


@pytest.mark.parametrize("sym", [False, True])
def test_every_scale_mantissa(sym):
    # group ranges over all fp16 mantissas and many exponents, on and next to rounding borders
    bits = torch.arange(0x0001, 0x7C00, 3, dtype=torch.int16).view(torch.float16)
    k = torch.zeros(bits.numel(), 1, 64, dtype=torch.float16)
    k[:, 0, 5] = bits
    k[:, 0, 40] = -bits
    k[:, 0, 41] = bits / 3
    gen = torch.Generator().manual_seed(5)
    k[:, 0, 8:30] = (bits[:, None].float() * (torch.rand(bits.numel(), 22, generator=gen) * 2 - 1)).half()
    n = bits.numel()
    cache = B.gq_kv4_empty(n // 64 + 1, 1, 64, 64, 32, sym)
    slots = torch.arange(n, device="cuda")
    B.gq_kv4_write(k.cuda(), k.cuda(), cache, slots, 32, sym)
    k32, v32 = B.gq_kv4_read(cache, slots, 64, 32, sym, torch.float32)
    want, _, _ = quantise64(k, 32, sym)
    assert torch.equal(k32.cpu().double(), want) and torch.equal(v32.cpu().double(), want)


def test_write_strided_skipped_and_nonfinite():
    gen = torch.Generator().manual_seed(3)
    t, hq, h, d, g = 21, 4, 2, 128, 64
    qkv = torch.randn(t, (hq + 2 * h) * d, generator=gen).to(torch.bfloat16)
    k = qkv[:, hq * d:(hq + h) * d].unflatten(1, (h, d))
    v = qkv[:, (hq + h) * d:].unflatten(1, (h, d))
    dev = qkv.cuda()
    kd = dev[:, hq * d:(hq + h) * d].unflatten(1, (h, d))
    vd = dev[:, (hq + h) * d:].unflatten(1, (h, d))
    assert not kd.is_contiguous()
    cache = B.gq_kv4_empty(4, h, d, 16, g, False)
    cache.zero_()
    slots = torch.arange(10, 10 + t)
    slots[3], slots[7], slots[9] = -1, 64, -(1 << 40)         # out of range: skipped, read as zeros
    B.gq_kv4_write(kd, vd, cache, slots.cuda(), g, False)
    k32, v32 = B.gq_kv4_read(cache, slots.cuda(), d, g, False, torch.float32)
    for got, x in ((k32, k), (v32, v)):
        want, _, _ = quantise64(x, g, False)
        want[[3, 7, 9]] = 0.0
        assert torch.equal(got.cpu().double(), want)
    same = torch.tensor([13, 17, 19], device="cuda")          # their slots stayed as they were
    k32, _ = B.gq_kv4_read(cache, same, d, g, False, torch.float32)
    assert not k32.any()
    bad = k.clone()
    bad[0, 0, 0], bad[1, 0, 0], bad[2, 0, 3] = math.inf, -math.inf, math.nan
    B.gq_kv4_write(bad.cuda(), bad.cuda(), cache, torch.arange(t).cuda(), g, False)
    k32, v32 = B.gq_kv4_read(cache, torch.arange(t).cuda(), d, g, False, torch.float32)
    assert torch.isfinite(k32).all() and torch.isfinite(v32).all()
    ok = torch.ones(t, h, d, dtype=torch.bool)
    ok[:3, 0, :g] = False                                     # only their groups are affected
    assert torch.equal(k32.cpu().double()[ok], quantise64(k, g, False)[0][ok])


class Problem:
    """A cache of random pages with poisoned memory around its tokens, and queries."""

    def __init__(self, seed, d, g, sym, page, dtype, h, r, q_lens, kv_lens, q_scale=1.5):
        gen = torch.Generator().manual_seed(seed)
        self.d, self.g, self.sym, self.page, self.dt = d, g, sym, page, DT[dtype]
        self.h, self.r, self.q_lens, self.kv_lens = h, r, q_lens, kv_lens
        need = [-(-n // page) for n in kv_lens]
        self.n_pages = sum(need) + 2
        perm = torch.randperm(self.n_pages, generator=gen).int()
        table = torch.full((len(need), max(need + [1]) + 1), 0x7FFFFFF0, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table = table
        slots = [table[b].long()[torch.arange(n) // page] * page + torch.arange(n) % page
                 for b, n in enumerate(kv_lens)]
        slots = torch.cat(slots) if slots else torch.zeros(0, dtype=torch.int64)
        t = sum(kv_lens)
        self.cache = B.gq_kv4_empty(self.n_pages, h, d, page, g, sym)
        fill_random(self.cache, gen)
        k, v = rows(gen, t, h, d, self.dt), rows(gen, t, h, d, self.dt)
        B.gq_kv4_write(k.cuda(), v.cuda(), self.cache, slots.cuda(), g, sym)
        self.k, sk, _ = quantise64(k, g, sym)
        self.v, sv, _ = quantise64(v, g, sym)
        self.sk, self.sv = sk.amax(-1), sv.amax(-1)
        self.q = (q_scale * torch.randn(sum(q_lens), h * r, d, generator=gen)).to(self.dt)
        self.starts = torch.tensor([0] + q_lens).cumsum(0).int()

    def run(self, q=None, table=None, kv_lens=None, starts="own", causal=True, window=0, scale=None, **kw):
        if isinstance(starts, str):
            starts = None if all(n == 1 for n in self.q_lens) else self.starts
        lens = torch.tensor(self.kv_lens if kv_lens is None else kv_lens, dtype=torch.int32)
        kw.setdefault("max_q_len", max(self.q_lens))
        kw.setdefault("max_kv_len", max(self.kv_lens))
        return B.gq_kv4_attention(
            self.q.cuda() if q is None else q, self.cache, (self.table if table is None else table).cuda(),
            lens.cuda(), self.g, self.sym, q_starts=None if starts is None else starts.cuda(), causal=causal,
            window=window, scale=scale, return_lse=True, **kw)

    def check(self, out, lse, causal=True, window=0, scale=None, dead=None, fp16_operands=False, what=""):
        scale = self.d ** -0.5 if scale is None else scale
        qa = ka = 0
        worst = worst_l = 0.0
        for b, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            q = self.q[qa:qa + n].double()
            k, v = self.k[ka:ka + kv], self.v[ka:ka + kv]
            o, l, p = attention64(q, k, v, n, kv, causal, window, scale, None if dead is None else dead[b])
            tol, ltol = attention_bounds(q, k, v, self.sk[ka:ka + kv], self.sv[ka:ka + kv], o, l, p, scale,
                                         self.dt, fp16_operands)
            got, gl = out[qa:qa + n].cpu().double(), lse[qa:qa + n].cpu().double()
            empty = l == -math.inf
            assert torch.equal(gl == -math.inf, empty), f"{what}: rows without keys, sequence {b}"
            assert not got[empty].any()
            if (~empty).any():
                worst = max(worst, float(((got - o).abs() / tol)[~empty].max()))
                worst_l = max(worst_l, float(((gl - l).abs() / ltol)[~empty].max()))
            assert torch.isfinite(got).all(), f"{what}: non-finite output, sequence {b}"
            qa, ka = qa + n, ka + kv
        announce(f"{what}: error / bound {worst:.3f}, lse {worst_l:.3f}")
        assert worst <= 1.0 and worst_l <= 1.0


def announce_case(p, what):
    announce(f"kv4 attention {what}: d={p.d} g={p.g} sym={p.sym} page={p.page} {p.dt} h={p.h} r={p.r} "
             f"q={p.q_lens} kv={p.kv_lens}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g,sym", LAYOUTS)
def test_single_tokens(d, g, sym, dtype):
    p = Problem(d * 3 + g, d, g, sym, 16, dtype, 2, 4, [1] * 8, [1, 0, 15, 16, 17, 33, 128, 201])
    announce_case(p, "single")
    p.check(*p.run(), what="single tokens")


@pytest.mark.parametrize("d,g,sym", LAYOUTS)
def test_long_split(d, g, sym):
    p = Problem(d + g, d, g, sym, 64, "bf16", 2, 2, [1] * 4, [2500, 3, 0, 1029])
    announce_case(p, "split")
    a = p.run()
    p.check(*a, what="split keys")
    b = p.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])     # no dependence on timing


@pytest.mark.parametrize("h,r", [(1, 1), (3, 7), (1, 64), (2, 8)])
@pytest.mark.parametrize("dtype,d,g", [("f16", 128, 64), ("bf16", 64, 64), ("bf16", 256, 128)])
def test_few_tokens_and_head_ratios(h, r, dtype, d, g):
    p = Problem(h * 10 + r, d, g, h == 3, 32, dtype, h, r, [4, 1, 6, 0, 2], [300, 1, 1400, 70, 9])
    announce_case(p, "few tokens")
    p.check(*p.run(), what="few tokens")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g,sym", LAYOUTS)
def test_prompts(d, g, sym, dtype):
    p = Problem(d * 5 + g, d, g, sym, 16, dtype, 2, 2, [150, 1, 0, 65, 200], [150, 40, 9, 1100, 333])
    announce_case(p, "prompts")
    a = p.run()
    p.check(*a, fp16_operands=True, what="prompts")
    b = p.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("h,r,q,kv", [(1, 64, [9, 70], [700, 70]), (3, 7, [40, 1, 80], [40, 1, 2000]),
                                      (8, 1, [513], [600])])
def test_prompt_head_ratios(h, r, q, kv):
    p = Problem(h + r, 128, 64, False, 64, "bf16", h, r, q, kv)
    announce_case(p, "prompt head ratios")
    p.check(*p.run(), fp16_operands=True, what="prompt head ratios")


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 20), (True, 130), (True, 2 ** 31 - 1)])
@pytest.mark.parametrize("long", [False, True])
def test_masks(causal, window, long):
    kv = [1500, 40, 9, 5, 2100] if long else [200, 40, 9, 5, 300]
    p = Problem(77 + window % 1000, 128, 32, False, 16, "f16", 2, 2, [70, 40, 12, 9, 1], kv)   # 12 > 9: rows before all keys
    announce_case(p, f"masks causal={causal} window={window}")
    p.check(*p.run(causal=causal, window=window), causal=causal, window=window, fp16_operands=True,
            what="masks")
    few = Problem(78 + window % 1000, 128, 32, False, 16, "f16", 2, 2, [7, 8, 3, 9, 1], kv)           # the other kernel
    few.check(*few.run(causal=causal, window=window), causal=causal, window=window, what="masks, few rows")


@pytest.mark.parametrize("max_kv", [None, 1, 5000])
def test_bounds_need_not_hold(max_kv):
    p = Problem(5, 128, 128, False, 16, "bf16", 2, 4, [9, 1, 30], [1300, 7, 45])
    announce_case(p, f"hints max_kv={max_kv}")
    for mq in (1, 30, 500):
        kw = dict(max_q_len=mq) if max_kv is None else dict(max_q_len=mq, max_kv_len=max_kv)
        p.check(*p.run(**kw), what=f"max_q_len={mq}", fp16_operands=mq > 1)


def test_bad_pages_and_lengths():
    p = Problem(9, 128, 64, False, 16, "bf16", 2, 4, [1, 3, 1], [100, 1200, 40])
    table = p.table.clone()
    table[0, 2], table[1, 70], table[1, 3] = -1, p.n_pages, -2 ** 31
    table[2, :] = 2 ** 31 - 1                                    # a sequence of bad pages only
    dead = [torch.zeros(n, dtype=torch.bool) for n in p.kv_lens]
    dead[0][32:48] = True
    dead[1][48:64] = True
    dead[1][1120:1136] = True
    dead[2][:] = True
    announce_case(p, "bad pages")
    p.check(*p.run(table=table), dead=dead, what="bad pages")
    for what, q_lens in (("few rows", [1, 3, 1]), ("many rows", [60, 70, 9])):
        p = Problem(19, 128, 64, False, 16, "bf16", 2, 4, q_lens, [100, 1200, 40])
        table = p.table.clone()
        table[0, 2], table[1, 70], table[1, 3] = -1, p.n_pages, -2 ** 31
        table[2, :] = 2 ** 31 - 1
        p.check(*p.run(table=table), dead=dead, fp16_operands=True, what="bad pages, " + what)
    # lengths below zero and beyond the table
    q = Problem(10, 128, 128, True, 16, "f16", 1, 2, [1, 1], [0, 64])
    short = q.table[:, :4].contiguous()
    out, lse = q.run(table=short, kv_lens=[-5, 1 << 30])
    q.check(out, lse, what="clamped lengths")


def test_query_starts_out_of_range_and_rows_left_alone():
    p = Problem(12, 64, 64, False, 16, "bf16", 2, 1, [2, 3], [50, 60])
    starts = torch.tensor([0, 2, 99], dtype=torch.int32)          # clamped to the 5 rows there are
    p.check(*p.run(starts=starts), what="clamped starts")
    out = torch.full((5, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    p.run(starts=torch.tensor([0, 2, 2], dtype=torch.int32), out=out)
    assert (out[2:] == 7.0).all() and not (out[:2] == 7.0).all()


def test_extreme_values():
    # scales over fp16's whole range, large scores, a key that takes all the weight
    for sk, sv, qs, q_lens in [(*c, n) for n in ([1, 2], [30, 50])
                               for c in ((1e-4, 1e-6, 2.0), (40.0, 3e4, 1.0), (1.0, 1e-7, 30.0), (1e-7, 60.0, 1e4))]:
        p = Problem(31, 128, 32, False, 16, "bf16", 1, 4, q_lens, [37, 1100], q_scale=qs)
        gen = torch.Generator().manual_seed(8)
        k, v = rows(gen, 1137, 1, 128, torch.bfloat16) * sk, rows(gen, 1137, 1, 128, torch.bfloat16) * sv
        slots = torch.cat([p.table[b].long()[torch.arange(n) // 16] * 16 + torch.arange(n) % 16
                           for b, n in enumerate(p.kv_lens)])
        B.gq_kv4_write(k.cuda(), v.cuda(), p.cache, slots.cuda(), 32, False)
        p.k, a, _ = quantise64(k, 32, False)
        p.v, b, _ = quantise64(v, 32, False)
        p.sk, p.sv = a.amax(-1), b.amax(-1)
        announce(f"kv4 extreme keys x{sk} values x{sv} queries x{qs}")
        p.check(*p.run(), fp16_operands=q_lens[0] > 1, what="extreme values")


def test_nonfinite_query_stays_in_its_row():
    for q_lens in ([1, 1], [40, 50]):
        p = Problem(14, 128, 128, False, 16, "bf16", 2, 4, q_lens, [70, 1300])
        q = p.q.cuda().clone()
        q[0, 1, 5], q[1, 6, 0] = math.nan, math.inf
        out, lse = p.run(q=q)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(out[1, 6]).all()
        ref, rl = p.run()
        keep = torch.ones(sum(q_lens), 8, dtype=torch.bool)
        keep[0, 1] = keep[1, 6] = False
        assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], rl[keep])


def test_strided_queries_streams_and_workspace():
    p = Problem(15, 128, 128, False, 16, "bf16", 2, 2, [1] * 6, [1500, 20, 64, 1, 900, 1100])
    ref, rl = p.run()
    p.check(ref, rl, what="plain strides")
    wide = torch.zeros(6, 8 * 128, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 256:256 + 512].unflatten(1, (4, 128))
    view.copy_(p.q)
    out, lse = p.run(q=view)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = p.run(q=view, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    need = B.gq_kv4_attention_workspace_size(6, 4, 2, 128, 1, 1500)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")     # of any content
    out, lse = p.run(workspace=ws)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    with pytest.raises(ValueError, match="workspace has"):
        p.run(workspace=ws[:need - 1])
    with pytest.raises(ValueError, match="passes the workspace"):
        p.run(stream=s.cuda_stream)


def test_graph_replays():
    p = Problem(16, 128, 64, False, 16, "bf16", 2, 4, [1] * 3, [1290, 30, 700])
    q, table = p.q.cuda(), p.table.cuda()
    lens = torch.tensor(p.kv_lens, dtype=torch.int32, device="cuda")
    k = torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([int(p.table[b, (n - 1) // 16]) * 16 + (n - 1) % 16
                          for b, n in enumerate(p.kv_lens)], device="cuda")

    def step():
        B.gq_kv4_write(k, k, p.cache, slots, 64, False)
        return B.gq_kv4_attention(q, p.cache, table, lens, 64, False, max_kv_len=1500)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        q.copy_(torch.randn_like(q))
        k.copy_(torch.randn_like(k))
        lens.copy_(torch.tensor([1290 - 300 * i, 30 - i, 700], dtype=torch.int32))
        g.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, step())


def test_empty_calls():
    cache = B.gq_kv4_empty(2, 2, 64, 16, 64)
    q = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    z = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    out, lse = B.gq_kv4_attention(q, cache, z, z[:, 0].contiguous(), 64, return_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    B.gq_kv4_write(q, q, cache, slots, 64)
    k, v = B.gq_kv4_read(cache, slots, 64, 64)
    assert k.shape == v.shape == (0, 2, 64)
    # no pages at all: every row is without keys
    q = torch.ones(3, 2, 64, dtype=torch.float16, device="cuda")
    out, lse = B.gq_kv4_attention(q, cache, torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                                  torch.ones(3, dtype=torch.int32, device="cuda"), 64, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()


def test_offsets_beyond_32_bits():
    # pages far beyond 4 GiB into the cache: 64-bit offsets
    h, d, page = 8, 128, 64
    n_pages = 80000                                              # 5.6 GB
    cache = B.gq_kv4_empty(n_pages, h, d, page, 128)
    assert cache.numel() > 1 << 32
    gen = torch.Generator().manual_seed(2)
    k, v = rows(gen, 200, h, d, torch.bfloat16), rows(gen, 200, h, d, torch.bfloat16)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2, 70000]], dtype=torch.int32)
    pos = torch.arange(200)
    slots = table[0].long()[pos // page] * page + pos % page
    B.gq_kv4_write(k.cuda(), v.cuda(), cache, slots.cuda())
    k32, v32 = B.gq_kv4_read(cache, slots.cuda(), d, out_dtype=torch.float32)
    assert torch.equal(k32.cpu().double(), quantise64(k, 128, False)[0])
    p = Problem(1, d, 128, False, page, "bf16", h, 1, [1], [200])
    p.cache, p.table = cache, table
    p.k, sk, _ = quantise64(k, 128, False)
    p.v, sv, _ = quantise64(v, 128, False)
    p.sk, p.sv = sk.amax(-1), sv.amax(-1)
    p.check(*p.run(), what="far pages")
