"""The choice of pages against its definition in 64 bits: the pages are equal, whole
number by whole number; then rotation, append, choice and attention together."""
import pytest
import torch

import kv8_util as U
from gpu_util import announce, device
from kv4_util import attention64
from test_gpu_kv8_store import DT, I32, draw, starts_of, tables
from test_gpu_rope import turn64
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu


def setup(h, d, page, dtype, kv_lens, seed=0):
    table, n_pages = tables(kv_lens, page, seed=seed)
    k = draw(sum(kv_lens), h, d, dtype, seed)
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device())
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, DT[dtype], device=device()).fill_(float("nan"))
    B.gq_kv8_append(k.to(device()), k.to(device()), cache, table.to(device()), I32(kv_lens), starts_of(kv_lens), bounds)
    return table, n_pages, k, cache, bounds


def check(q, bounds, table, q_lens, kv_lens, page, keep, first, last, h, dead=(), n_pages=None, **kw):
    single = all(n == 1 for n in q_lens)
    pages, lens = B.gq_kv8_select(q.to(device()), bounds, table.to(device()), I32(kv_lens), keep, page,
                                  q_starts=None if single else starts_of(q_lens), first=first, last=last, **kw)
    torch.cuda.synchronize()
    pages, lens, bd, at = pages.cpu(), lens.cpu(), bounds.cpu().double(), 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        for i in range(n):
            p = kv - n + i
            want = torch.full((h, keep), -1, dtype=torch.int32)
            seen = 0
            if p >= 0:
                row = table[b, :p // page + 1].long()
                safe = row.clamp(0, bd.shape[0] - 1)
                gone = [j for j, x in enumerate(row.tolist()) if x < 0 or x >= bd.shape[0]]
                sel, seen = U.select64(q[at].double(), bd[safe, :, 0], bd[safe, :, 1], p, page, keep, first, last, gone)
                for x in range(h):
                    want[x, :len(sel[x])] = table[b, sel[x]]
            assert int(lens[at]) == seen
            assert torch.equal(pages[at], want), f"sequence {b}, query {i}"
            at += 1
    return pages, lens


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,h,d,page,q_lens,kv_lens,keep,first,last", [
    (8, 2, 128, 16, [1, 1, 1], [1000, 16, 3], 8, 1, 1), (4, 4, 64, 32, [3, 1, 2], [700, 33, 2], 5, 0, 2),
    (6, 2, 96, 16, [1, 4], [500, 90], 7, 2, 1), (3, 1, 256, 64, [1, 1], [3000, 64 * 9], 9, 1, 3),
    (64, 1, 64, 16, [2], [800], 30, 1, 1), (2, 1, 128, 16, [1], [1300], 1, 0, 1), (2, 1, 128, 16, [1], [1300], 4, 2, 2),
    (2, 2, 64, 16, [1, 1], [4000, 1], 249, 1, 1), (2, 2, 64, 16, [1], [4000], 250, 1, 1), (4, 1, 128, 1024, [2], [5000], 3, 1, 1)])
def test_choice(dtype, hq, h, d, page, q_lens, kv_lens, keep, first, last):
    announce(f"select {dtype} {hq}/{h}x{d} page {page} {q_lens} {kv_lens} keep {keep}")
    table, n_pages, k, cache, bounds = setup(h, d, page, dtype, kv_lens)
    q = torch.randn(sum(q_lens), hq, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    check(q, bounds, table, q_lens, kv_lens, page, keep, first, last, h)
    check(q, bounds, table, q_lens, kv_lens, page, keep, first, last, h, max_kv_len=max(kv_lens))


def test_ties_and_scores_close_together():
    """Equal pages go to the earlier one; scores that differ by one part in 2^40 are told apart."""
    h, d, page, n = 1, 64, 16, 300
    table, n_pages = tables([n * page], page)
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, torch.float16, device=device()).zero_()
    q = torch.zeros(1, 1, d)
    q[0, 0, 0], q[0, 0, 1] = 1.0, 2.0 ** -12
    tb = table[0].long()
    for pattern in range(4):
        lo = torch.zeros(n_pages, h, 2, d)
        if pattern == 1:                       # two values
            lo[tb[torch.arange(0, n, 3)], 0, :, 0] = 1.0
        if pattern == 2:                       # 1024 and n 2^-36 beside it
            lo[tb, 0, :, 0] = 1024.0
            lo[tb, 0, :, 1] = ((torch.arange(n) * 37) % n).float()[:, None] * 2.0 ** -24
        if pattern == 3:                       # negative, zeros of both signs among them
            lo[tb, 0, :, 0] = -((torch.arange(n) * 7) % 11).float()[:, None]
        bounds.copy_(lo)
        for keep in (2, 17, 100, 299):
            check(q.half(), bounds, table, [1], [n * page], page, keep, 1, 1, h)


def test_pages_that_do_not_exist_and_values_that_are_not_finite():
    h, d, page = 2, 64, 16
    table, n_pages, k, cache, bounds = setup(h, d, page, "bf16", [640], seed=3)
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    table[0, 5], table[0, 9], table[0, 20] = -1, n_pages, 1 << 30
    for keep in (6, 37, 38, 39):
        check(q, bounds, table, [1], [640], page, keep, 1, 1, h)
    q[0, 1, 3] = float("nan")                   # its sums do not count, those of the heads beside it do
    check(q, bounds, table, [1], [640], page, 6, 1, 1, h)
    q[0, 0, 3] = float("nan")                   # a group without sums: the earliest pages
    pages, _ = check(q, bounds, table, [1], [640], page, 6, 1, 1, h)
    assert pages[0, 0].tolist() == table[0, [0, 1, 2, 3, 4, 39]].tolist()


def test_scores_that_are_infinite():
    """Scores of both infinities and between them, pages that do not exist among them: the
    whole range of the scores' integers."""
    h, d, page, n = 1, 64, 16, 300
    table, n_pages = tables([n * page], page)
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, torch.bfloat16, device=device())
    q = torch.zeros(1, 2, d).bfloat16()
    q[0, 0, 0], q[0, 0, 1], q[0, 1, 1] = float("inf"), 1.0, 2.0 ** 100
    g = torch.Generator().manual_seed(6)
    for every in (2, 7, 150):
        lo = torch.randn(n_pages, h, 2, d, generator=g).sort(2).values      # smallest, largest
        up = torch.arange(n) % every == 1
        lo[table[0].long(), 0, :, 0] = torch.where(up, 1.0, -1.0)[:, None]
        bounds.copy_(lo)
        for keep in (2, 3, 17, 100, 299):
            check(q[:, :1], bounds, table, [1], [n * page], page, keep, 1, 1, h)      # +inf and -inf alone
            check(q, bounds, table, [1], [n * page], page, keep, 1, 1, h)             # and finite ones
            gone = table.clone()
            gone[0, 3::5] = -1
            check(q, bounds, gone, [1], [n * page], page, keep, 1, 1, h)


def test_queries_without_pages_and_lengths_out_of_range():
    h, d, page = 2, 64, 16
    table, n_pages, k, cache, bounds = setup(h, d, page, "bf16", [100, 40], seed=4)
    q = torch.randn(8, 4, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    # more queries than keys, rows behind the last sequence
    pages, lens = B.gq_kv8_select(q.to(device()), bounds, table.to(device()), I32([2, 40]), 3, page, q_starts=I32([0, 4, 6]))
    assert lens.tolist() == [0, 0, 1, 2, 39, 40, 0, 0]
    assert bool((pages[[0, 1, 6, 7]] == -1).all()) and pages[2, 0].tolist() == [int(table[0, 0]), -1, -1]
    pages, lens = B.gq_kv8_select(q[:2].to(device()), bounds, table.to(device()), I32([-3, 10000]), 3, page)
    assert lens.tolist() == [0, 48] and bool((pages[0] == -1).all())      # the table holds 7 pages: 112 of 10000
    # a bound that is too small: lengths count as that many, rounded up to whole pages
    pages, lens = B.gq_kv8_select(q[:2].to(device()), bounds, table.to(device()), I32([100, 40]), 3, page, max_kv_len=33)
    want, seen = B.gq_kv8_select(q[:2].to(device()), bounds, table.to(device()), I32([48, 40]), 3, page)
    assert torch.equal(lens, seen) and torch.equal(pages, want) and lens.tolist() == [48, 40]
    pages, lens = B.gq_kv8_select(q[:2].to(device()), bounds, table[:, :0].contiguous().to(device()), I32([5, 5]), 3, page)
    assert lens.tolist() == [0, 0] and bool((pages == -1).all())
    pages, lens = B.gq_kv8_select(q[:0].to(device()), bounds, table[:0].to(device()), I32([]), 3, page)
    assert pages.shape == (0, h, 3) and lens.shape == (0,)


def test_long_table():
    """More pages than are kept in LDS while they are sorted out."""
    h, d, page, n = 1, 64, 16, 9001
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2)).int()[None]
    g = torch.Generator(device=device()).manual_seed(3)
    bounds = torch.randn(n, h, 2, d, generator=g, device=device()).sort(2).values.bfloat16()
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    for keep in (2, 64, 3001):
        check(q, bounds, table, [1], [n * page - 5], page, keep, 1, 1, h)


def test_everything_kept_is_dense_attention():
    h, d, page = 2, 128, 16
    table, n_pages, k, cache, bounds = setup(h, d, page, "bf16", [300, 45], seed=5)
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(device())
    tb, lens = table.to(device()), I32([300, 45])
    pages, seen = B.gq_kv8_select(q, bounds, tb, lens, 19, page)
    assert torch.equal(seen, lens) and torch.equal(pages[:, 0, :19], tb) and torch.equal(pages[:, 1], tb)
    assert torch.equal(B.gq_kv8_attention(q, cache, pages, seen, max_kv_len=300), B.gq_kv8_attention(q, cache, tb, lens, max_kv_len=300))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_step_together(dtype):
    """Prompts of three sequences, then single tokens captured into a graph: rotation, append,
    choice and attention in a run, each against its definition."""
    hq, h, d, page, keep, dt = 8, 2, 128, 16, 4, DT[dtype]
    prompts, steps = [90, 17, 140], 6
    table, n_pages = tables([n + steps for n in prompts], page)
    tb = table.to(device())
    f, m = B.gq_rope_frequencies(64, 10000.0, "yarn", factor=4.0, original_length=64, low=1.0, high=32.0, device=device())
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device())
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, dt, device=device())
    g = torch.Generator().manual_seed(0)
    new = lambda n: torch.randn(n, hq + 2 * h, d, generator=g).to(dt)
    qkv = new(sum(prompts)).to(device())
    pos = torch.cat([torch.arange(n) for n in prompts]).to(device())
    lens = I32(prompts)
    turned = B.gq_rope(qkv[:, :hq + h], pos, f, amplitude=m)
    B.gq_kv8_append(turned[:, hq:], qkv[:, hq + h:], cache, tb, lens, starts_of(prompts), bounds)
    out = B.gq_kv8_attention(turned[:, :hq], cache, tb, lens, starts_of(prompts), max(prompts), max(prompts))
    keys, vals, cuts, at = [], [], [[n] for n in prompts], 0
    for b, n in enumerate(prompts):
        y, size = turn64(qkv[at:at + n, :hq + h].cpu(), pos[at:at + n].cpu(), f.cpu(), False, m, False)
        got = turned[at:at + n].cpu()
        assert bool(((got.double() - y).abs() <= torch.finfo(dt).eps / 2 * y.abs() + 2.0 ** -19 * m * size + 2.0 ** -25).all())
        keys.append(got[:, hq:])
        vals.append(qkv[at:at + n, hq + h:].cpu())
        compare(out[at:at + n], got[:, :hq], keys[b], vals[b], cuts[b], n, dt)
        at += n

    x, p1, l1 = new(3).to(device()), lens.long(), lens + 1
    state = {}

    def step():
        t = B.gq_rope(x[:, :hq + h], p1, f, amplitude=m)
        B.gq_kv8_append(t[:, hq:], x[:, hq + h:], cache, tb, l1, None, bounds)
        pages, seen = B.gq_kv8_select(t[:, :hq], bounds, tb, l1, keep, page, max_kv_len=max(prompts) + steps)
        state.update(t=t, pages=pages, seen=seen, out=B.gq_kv8_attention(t[:, :hq], cache, pages, seen))
    step()                  # the first token, and what is set up once
    torch.cuda.synchronize()
    record(state, x, keys, vals, cuts, hq, h, table, bounds, page, keep, dt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, steps):
        x.copy_(new(3))
        p1 += 1
        l1 += 1
        graph.replay()
        torch.cuda.synchronize()
        record(state, x, keys, vals, cuts, hq, h, table, bounds, page, keep, dt)


def record(state, x, keys, vals, cuts, hq, h, table, bounds, page, keep, dt):
    """Take the step's tokens over into the reference and compare what it gave."""
    t, v, bd = state["t"].cpu(), x[:, hq + h:].cpu(), bounds.cpu().double()
    for b in range(3):
        keys[b] = torch.cat((keys[b], t[b:b + 1, hq:]))
        vals[b] = torch.cat((vals[b], v[b:b + 1]))
        n = keys[b].shape[0]
        cuts[b].append(n)
        row = table[b, :(n - 1) // page + 1].long()
        for j in range(row.numel()):
            part = keys[b][j * page:(j + 1) * page].double()
            assert torch.equal(bd[row[j], :, 0], part.amin(0)) and torch.equal(bd[row[j], :, 1], part.amax(0))
        sel, seen = U.select64(t[b, :hq].double(), bd[row, :, 0], bd[row, :, 1], n - 1, page, keep, 1, 1)
        assert int(state["seen"][b]) == seen
        for y in range(h):
            assert state["pages"][b, y, :len(sel[y])].tolist() == table[b, sel[y]].tolist()
        compare(state["out"][b:b + 1], t[b:b + 1, :hq], keys[b], vals[b], cuts[b], 1, dt, sel, page)


def compare(out, q, k, v, cuts, n, dt, sel=None, page=None):
    kk, sk = U.cached(k, cuts[:-1])
    vv, sv = U.cached(v, cuts[:-1])
    r, d = q.shape[1] // k.shape[1], q.shape[2]
    for h in range(k.shape[1]):
        keep = torch.arange(k.shape[0]) if sel is None else \
            torch.cat([torch.arange(j * page, min((j + 1) * page, k.shape[0])) for j in sel[h]])
        a = [t[keep, h:h + 1] for t in (kk, vv, sk, sv)]
        qh = q[:, h * r:(h + 1) * r].double()
        o, l, p = attention64(qh, a[0], a[1], n, keep.numel(), True, 0, d ** -0.5)
        tol, _ = U.attention_bounds(qh, *a, o, l, p, d ** -0.5, dt, False)
        assert bool(((out[:, h * r:(h + 1) * r].cpu().double() - o).abs() <= tol).all())


def test_infinite_queries_beside_bounds_of_zero():
    """The product with the bound that does not count is not formed: infinity times 0 makes NaN only
    of pages where it does."""
    h, d, page, n = 1, 64, 16, 60
    table, n_pages = tables([n * page], page)
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, torch.bfloat16, device=device())
    lo = torch.zeros(n_pages, h, 2, d)
    rows = table[0].long()
    lo[rows[0::3], 0, 1] = 5.0                       # 0 .. 5
    lo[rows[1::3], 0, 0] = -5.0                      # -5 .. 0
    lo[rows[2::3], 0, 0], lo[rows[2::3], 0, 1] = -1.0, 2.0
    bounds.copy_(lo)
    first = lambda which, skip: [j for j in range(which, n, 3) if j not in skip]
    for sign, best, nan in ((1.0, (0, 2), 1), (-1.0, (1, 2), 0)):
        q = torch.zeros(1, 1, d).bfloat16()
        q[0, 0, 7] = sign * float("inf")
        for keep in (10, 45):
            pages, lens = B.gq_kv8_select(q.to(device()), bounds, table.to(device()), I32([n * page]), keep, page)
            order = sorted(first(best[0], (0, n - 1)) + first(best[1], (0, n - 1))) + first(nan, (0, n - 1))
            want = sorted([0, n - 1] + order[:keep - 2])
            assert pages[0, 0].tolist() == table[0, want].tolist() and int(lens[0]) == keep * page
