"""Appending to the 8-bit cache and reading it back, bit for bit: codes, scales and
bounds are exact (one rounding each, in a defined order), so the values read in fp32
equal fl32(S q) and 16-bit ones that rounded again."""
import pytest
import torch

import kv8_util as U
from gpu_util import announce, device
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
I32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device())


def tables(lens, page, spare=2, seed=0, width=None):
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).int()
    t = torch.full((len(lens), width or max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, n_pages


def slots_of(table, b, n, page):
    pos = torch.arange(n)
    return table[b, pos // page].long() * page + pos % page


def starts_of(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return I32(out)


def draw(n, h, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, d, generator=g) * torch.exp(2 * torch.randn(n, h, 1, generator=g))
    if n * h:
        x[..., 0] *= 7
        x[torch.rand(n, h, generator=g) < 0.05] = 0
    return x.to(DT[dtype])


def expect(x, cuts, dtype):
    """Values of one sequence as fp32 and as the 16-bit type."""
    v, _ = U.cached(x, cuts)
    v = v.float()
    return v, v.to(DT[dtype])


def read_all(cache, table, lens, page, d, out):
    slots = torch.cat([slots_of(table, b, n, page) for b, n in enumerate(lens)]).to(device())
    return B.gq_kv8_read(cache, slots, d, out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,h,page", [(64, 3, 16), (96, 2, 32), (128, 8, 64), (256, 1, 16), (128, 1, 1024)])
def test_appends(dtype, d, h, page):
    """Three sequences grow by calls of uneven lengths (none, one, odd, across pages)."""
    calls = [(5, 0, 40), (0, 1, 1), (11, 17, 1), (1, 1, 1), (33, 16, 100), (1, 0, 2 * page + 3), (2, 3, 5)]
    total = [sum(c[b] for c in calls) for b in range(3)]
    announce(f"append {dtype} d={d} h={h} page={page} totals {total}")
    table, n_pages = tables(total, page)
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device()).fill_(0xFF)
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, DT[dtype], device=device()).fill_(float("nan"))
    k, v = [draw(n, h, d, dtype, 10 + b) for b, n in enumerate(total)], [draw(n, h, d, dtype, 20 + b) for b, n in enumerate(total)]
    at, cuts = [0, 0, 0], [[], [], []]
    for c in calls:
        part = lambda xs: torch.cat([x[a:a + n] for x, a, n in zip(xs, at, c)]).to(device())
        kk, vv = part(k), part(v)
        at = [a + n for a, n in zip(at, c)]
        B.gq_kv8_append(kk, vv, cache, table.to(device()), I32(at), starts_of(c), bounds)
        for b in range(3):
            cuts[b].append(at[b])
        torch.cuda.synchronize()
    gk, gv = read_all(cache, table, total, page, d, torch.float32)
    hk, hv = read_all(cache, table, total, page, d, DT[dtype])
    for got, half, xs in ((gk, hk, k), (gv, hv, v)):
        want = [expect(x, c, dtype) for x, c in zip(xs, cuts)]
        assert torch.equal(got.cpu(), torch.cat([w[0] for w in want]))
        assert torch.equal(half.cpu(), torch.cat([w[1] for w in want]))
    for b, n in enumerate(total):
        for j in range(-(-n // page)):
            part = k[b][j * page:(j + 1) * page]
            got = bounds[table[b, j]].cpu()
            assert torch.equal(got[:, 0], part.amin(0)) and torch.equal(got[:, 1], part.amax(0))


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_single_tokens(d):
    """Token by token without starts: each call requantises what the block holds."""
    h, page, n = 2, 16, 37
    table, n_pages = tables([n, n], page)
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device()).fill_(0xFF)
    k, v = [draw(n, h, d, "bf16", 1 + b) for b in range(2)], [draw(n, h, d, "bf16", 5 + b) for b in range(2)]
    for t in range(n):
        B.gq_kv8_append(torch.stack([x[t] for x in k]).to(device()), torch.stack([x[t] for x in v]).to(device()), cache,
                        table.to(device()), I32([t + 1, t + 1]))
    gk, gv = read_all(cache, table, [n, n], page, d, torch.float32)
    for got, xs in ((gk, k), (gv, v)):
        assert torch.equal(got.cpu(), torch.cat([expect(x, list(range(1, n)), "bf16")[0] for x in xs]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_borders_of_rounding(dtype):
    """Values at and next to k + 1/2 steps: S is a power of two, so 16-bit values hit them."""
    d = 64
    x = torch.zeros(16, 1, d)
    x[0, 0, 0] = 127.0
    for i in range(16):
        x[i, 0, 1:33] = torch.arange(32) + 0.5 + i * 3
        x[i, 0, 33:] = -(torch.arange(31) + 0.5 + i * 3)
    for shift, scale in enumerate((1.0, 0.5, 2.0 ** -9, 3.0)):
        y = (x * scale).to(DT[dtype])
        y[5, 0, 3] = torch.nextafter(y[5, 0, 3].float(), torch.tensor(0.0)).to(DT[dtype])
        table, n_pages = tables([16], 16)
        cache = B.gq_kv8_empty(n_pages, 1, d, 16, device=device())
        B.gq_kv8_append(y.to(device()), -y.to(device()), cache, table.to(device()), I32([16]), I32([0, 16]))
        gk, gv = read_all(cache, table, [16], 16, d, torch.float32)
        assert torch.equal(gk.cpu(), expect(y, [], dtype)[0]) and torch.equal(gv.cpu(), expect(-y, [], dtype)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_ends_of_the_range(dtype):
    """Zeros, values far below the least step, the type's largest, infinities, NaN."""
    d, big = 64, float(torch.finfo(DT[dtype]).max)
    x = torch.zeros(6 * 16, 1, d)
    x[16:32] = 2.0 ** -24 if dtype == "f16" else 2.0 ** -60
    x[32:48] = torch.linspace(-1, 1, 64) * big
    x[48:64] = torch.linspace(-1, 1, 64)
    x[50, 0, 3], x[51, 0, 4], x[52, 0, 5] = float("inf"), float("-inf"), float("nan")
    x[64:80, 0, ::2] = float("nan")
    x[80:] = 2.0 ** -14
    y = x.to(DT[dtype])
    table, n_pages = tables([96], 32)
    cache = B.gq_kv8_empty(n_pages, 1, d, 32, device=device()).fill_(0xFF)
    bounds = B.gq_kv8_bounds_empty(n_pages, 1, d, DT[dtype], device=device())
    B.gq_kv8_append(y.to(device()), y.to(device()), cache, table.to(device()), I32([96]), I32([0, 96]), bounds)
    gk, gv = read_all(cache, table, [96], 32, d, torch.float32)
    want = expect(y, [], dtype)[0]
    assert torch.equal(gk.cpu(), want) and torch.equal(gv.cpu(), want)
    clean = torch.nan_to_num(y.float(), nan=0.0, posinf=big, neginf=-big).to(DT[dtype])
    for j in range(3):
        got = bounds[table[0, j]].cpu()
        assert torch.equal(got[:, 0], clean[32 * j:32 * j + 32].amin(0)) and torch.equal(got[:, 1], clean[32 * j:32 * j + 32].amax(0))


def test_views_and_bytes_left_alone():
    """k and v as slices of a fused projection; slots, bounds and rows that a call does not
    name keep their content; tokens without a page are skipped."""
    d, h, page = 128, 2, 16
    qkv = draw(50, 8, d, "bf16", 3).to(device())
    k, v = qkv[:, 4:6], qkv[:, 6:8]
    lens, new = [20, 40, 3, 33], [20, 7, 10, 5]      # the third begins before its sequence does
    table, n_pages = tables([20, 40, 16, 48], page, spare=3)
    table[1, 2] = n_pages + 5                        # no such page: positions 32 .. 39 of sequence 1
    table[3] = -1                                    # no pages at all
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device()).fill_(0x5A)
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, device=device()).fill_(9.0)
    rows = sum(new)
    B.gq_kv8_append(k, v, cache, table.to(device()), I32(lens), starts_of(new), bounds)
    torch.cuda.synchronize()
    at = 27 + 7                                      # the third's last three tokens
    for got, x in ((0, k.cpu()), (1, v.cpu())):
        g = B.gq_kv8_read(cache, slots_of(table, 0, 20, page).to(device()), d, torch.float32)[got]
        assert torch.equal(g.cpu(), expect(x[:20], [], "bf16")[0])
        g = B.gq_kv8_read(cache, slots_of(table, 2, 3, page).to(device()), d, torch.float32)[got]
        assert torch.equal(g.cpu(), expect(x[at:at + 3], [], "bf16")[0])
    used = [int(table[0, 0]), int(table[0, 1]), int(table[2, 0])]
    rest = [p for p in range(n_pages) if p not in used]
    flat = cache.view(-1)
    codes = flat[:n_pages * h * page * 2 * d].view(n_pages, -1)
    scales = flat[n_pages * h * page * 2 * d:].view(n_pages, -1)
    assert bool((codes[rest] == 0x5A).all()) and bool((scales[rest] == 0x5A).all())
    assert bool((bounds[rest] == 9.0).all())
    assert rows == 42                                # rows 42 .. 49 belong to nobody


def test_past_the_table_and_empty_calls():
    d, page = 64, 16
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=device())
    cache = B.gq_kv8_empty(2, 1, d, page, device=device()).fill_(0x11)
    x = draw(10, 1, d, "f16", 1).to(device())
    B.gq_kv8_append(x, x, cache, table, I32([38]), I32([0, 10]))     # positions 28 .. 37 of 32
    got = B.gq_kv8_read(cache, torch.arange(12, 16, device=device()), d, torch.float32)[0]
    b = U.Blocks(d)
    b.codes, b.scales = torch.zeros(12, d, dtype=torch.float64), [0.0]
    before = cache.clone()
    B.gq_kv8_append(x[:0], x[:0], cache, table, I32([38]), I32([0, 0]))
    B.gq_kv8_append(x[:0], x[:0], cache, table[:0], I32([]))
    B.gq_kv8_append(x, x, cache, table[:, :0].contiguous(), I32([10]), I32([0, 10]))
    assert torch.equal(cache, before)
    # older tokens 16 .. 27 hold a scale of 0x11111111 (1e-28): the new ones' own prevails
    want = x[:4, 0].cpu().double()
    s = U.scale_of(want)
    assert torch.equal(got[:, 0].cpu(), (torch.round(want / s) * s).float())
    k, v = B.gq_kv8_read(cache, torch.tensor([-1, 32, 1 << 40], device=device()), d)
    assert not k.any() and not v.any()
    assert B.gq_kv8_read(cache, torch.zeros(0, dtype=torch.int64, device=device()), d)[0].shape == (0, 1, d)


def test_cut_back_and_pages_used_again():
    """A sequence that loses tokens and is appended to keeps the scale and bounds of the block
    and page it was cut in; a page that is begun anew does not."""
    d, page = 64, 32
    k = draw(64, 1, d, "bf16", 8)
    k[20:30] *= 50
    new = draw(20, 1, d, "bf16", 9)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=device())
    cache = B.gq_kv8_empty(2, 1, d, page, device=device())
    bounds = B.gq_kv8_bounds_empty(2, 1, d, device=device())
    app = lambda x, end: B.gq_kv8_append(x.to(device()), x.to(device()), cache, table, I32([end]), I32([0, x.shape[0]]), bounds)
    app(k, 64)
    app(new, 42)                                     # positions 22 .. 41: cut back to 22
    got = read_all(cache, table.cpu(), [42], page, d, torch.float32)[0]
    b = U.Blocks(d).append(k[:22, 0])
    b.scales[1] = max(b.scales[1], U.scale_of(k[16:32, 0]))
    b.codes[16:] = torch.round(k[16:22, 0].double() / b.scales[1])
    b.append(new[:, 0])
    assert torch.equal(got[:, 0].cpu(), b.values().float())
    wide = torch.cat((k[:32], new[:10])).float()
    assert torch.equal(bounds[1, 0, 0].cpu().float(), wide.amin((0, 1)))
    assert torch.equal(bounds[0, 0, 1].cpu().float(), new[10:, 0].float().amax(0))


def test_many_sequences_and_long_prompts():
    """Sequences found among many, empty ones in between; a run of 16 input rows that holds
    several sequences; 3000 tokens of one."""
    d, h, page = 64, 2, 16
    lens = [(i * 7) % 4 for i in range(700)] + [3000] + [0, 0, 1]
    table, n_pages = tables(lens, page, width=190)
    k = draw(sum(lens), h, d, "bf16", 4)
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device())
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, device=device())
    for batch in (len(lens), 704 - 3):               # few and many tokens a sequence
        first = len(lens) - batch
        n = sum(lens[first:])
        x = k[k.shape[0] - n:].to(device())
        cache.fill_(0xFF)
        B.gq_kv8_append(x, -x, cache, table[first:].contiguous().to(device()), I32(lens[first:]), starts_of(lens[first:]), bounds)
        gk, gv = read_all(cache, table[first:], lens[first:], page, d, torch.float32)
        want, at = [], 0
        for m in lens[first:]:
            want.append(expect(k[k.shape[0] - n + at:k.shape[0] - n + at + m], [], "bf16")[0])
            at += m
        want = torch.cat(want)
        assert torch.equal(gk.cpu(), want) and torch.equal(gv.cpu(), -want)
    long = [p for p in table[700].tolist() if p >= 0]
    at = sum(lens[:700])
    for j in (0, 17, 187):
        part = k[at + 16 * j:min(at + 3000, at + 16 * j + 16)]
        assert torch.equal(bounds[long[j]].cpu()[:, 0], part.amin(0))


@pytest.mark.parametrize("page,lens", [(32, [1111, 40, 1700]), (64, [2053, 700, 31]), (128, [1025, 2000]), (256, [4097])])
def test_long_prompts_in_pages_of_several_blocks(page, lens):
    """Every block and every bound of prompts that fill the dies several times over."""
    d, h = 64, 2
    table, n_pages = tables(lens, page, seed=page)
    k = draw(sum(lens), h, d, "bf16", 9)
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device()).fill_(0xFF)
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, device=device()).fill_(float("nan"))
    x = k.to(device())
    B.gq_kv8_append(x, -x, cache, table.to(device()), I32(lens), starts_of(lens), bounds)
    gk, gv = read_all(cache, table, lens, page, d, torch.float32)
    bounds, at = bounds.cpu(), 0
    for b, n in enumerate(lens):
        want = expect(k[at:at + n], [], "bf16")[0]
        assert torch.equal(gk[at:at + n].cpu(), want) and torch.equal(gv[at:at + n].cpu(), -want)
        for j in range(-(-n // page)):
            part = k[at + page * j:at + min(n, page * j + page)]
            got = bounds[table[b, j].long()]
            assert torch.equal(got[:, 0], part.amin(0)) and torch.equal(got[:, 1], part.amax(0))
        at += n


def test_graph_and_stream():
    d, h, page = 128, 2, 16
    table, n_pages = tables([64], page)
    tb = table.to(device())
    x = torch.zeros(1, h, d, dtype=torch.bfloat16, device=device())
    lens = I32([1])
    cache = B.gq_kv8_empty(n_pages, h, d, page, device=device())
    bounds = B.gq_kv8_bounds_empty(n_pages, h, d, device=device())
    B.gq_kv8_append(x, x, cache, tb, lens, None, bounds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gq_kv8_append(x, x, cache, tb, lens, None, bounds)
    data = draw(40, h, d, "bf16", 2)
    for t in range(40):
        x.copy_(data[t:t + 1])
        lens.fill_(t + 1)
        graph.replay()
    torch.cuda.synchronize()
    want = expect(data, list(range(1, 40)), "bf16")[0]
    assert torch.equal(read_all(cache, table, [40], page, d, torch.float32)[0].cpu(), want)
    other = B.gq_kv8_empty(n_pages, h, d, page, device=device())
    s = torch.cuda.Stream()
    data, start = data.to(device()), I32([0, 40])
    s.wait_stream(torch.cuda.current_stream())
    n40 = I32([40])
    B.gq_kv8_append(data, data, other, tb, n40, start, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(read_all(other, table, [40], page, d, torch.float32)[1].cpu(), expect(data.cpu(), [], "bf16")[0])
