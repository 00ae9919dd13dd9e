"""Storage of the 4-bit cache: which bytes a write touches, and calls that take
more than one launch."""
import pytest
import torch

from gpu_util import announce
from test_gpu_kv4 import DT, LAYOUTS, rows
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g,sym", LAYOUTS)
def test_write_touches_its_tokens_alone(d, g, sym, dtype):
    # Bytes that two caches of different content hold alike after the same write
    # were written; all others kept their content.  A token owns a row's bytes.
    gen = torch.Generator().manual_seed(d * 13 + g)
    t, h, page, n_pages = 45, 3, 32, 5
    announce(f"kv4 bytes written d={d} g={g} sym={sym} {dtype}")
    k, v = rows(gen, t, h, d, DT[dtype]).cuda(), rows(gen, t, h, d, DT[dtype]).cuda()
    slots = torch.randperm(n_pages * page, generator=gen)[:t]
    slots[4], slots[11], slots[12] = -1, n_pages * page, -(1 << 33)
    after = []
    for byte in (0x00, 0xFF):
        cache = B.gq_kv4_empty(n_pages, h, d, page, g, sym)
        cache.fill_(byte)
        B.gq_kv4_write(k, v, cache, slots.cuda(), g, sym)
        after.append(cache.cpu())
    written = after[0] == after[1]
    assert not after[0][~written].any() and (after[1][~written] == 0xFF).all()
    row = d // 2 + (2 if sym else 4) * (d // g)
    assert int(written.sum()) == 2 * (t - 3) * h * row


def test_storage_calls_of_more_than_one_launch():
    # 2^24 tokens go into one launch; rows overlap in memory (a token stride of 8
    # elements), so each token's is its own and the next launch's differ
    top, d, page, n_pages = 1 << 24, 64, 64, 40
    t = top + 40
    announce(f"kv4 storage of {t} tokens")
    gen = torch.Generator(device="cuda").manual_seed(17)
    base = torch.randn(8 * t + d, generator=gen, device="cuda").to(torch.float16)
    k = base.as_strided((t, 1, d), (8, d, 1))
    v = base.flip(0).as_strided((t, 1, d), (8, d, 1))
    cache = B.gq_kv4_empty(n_pages, 1, d, page, 32)
    cache.zero_()
    slots = torch.full((t,), -1, dtype=torch.int64, device="cuda")
    some = torch.cat([torch.arange(30), torch.arange(top - 40, t)]).cuda()
    places = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(1))[:some.numel()].cuda()
    slots[some] = places
    B.gq_kv4_write(k, v, cache, slots, 32)
    # the same tokens in one launch
    want = torch.zeros_like(cache)
    B.gq_kv4_write(k[some], v[some], want, places, 32)
    assert torch.equal(cache, want)
    # read back: every slot again and again, both launches
    every = torch.arange(n_pages * page, device="cuda")
    kw, vw = B.gq_kv4_read(cache, every, d, 32, out_dtype=torch.float16)
    slots = torch.arange(t, device="cuda") * 7 % (n_pages * page)
    slots[top - 1], slots[top + 1] = -1, n_pages * page
    ok = (slots >= 0) & (slots < n_pages * page)
    ko, vo = B.gq_kv4_read(cache, slots, d, 32, out_dtype=torch.float16)
    for got, ref in ((ko, kw), (vo, vw)):
        for a in range(0, t, 1 << 22):
            b = min(t, a + (1 << 22))
            assert torch.equal(got[a:b], ref[slots[a:b].clamp(0, n_pages * page - 1)] * ok[a:b, None, None])


@pytest.mark.parametrize("d,g,sym,h", [(64, 32, True, 8), (96, 96, False, 8), (128, 64, False, 8), (256, 32, False, 4)])
def test_results_past_the_last_cache(d, g, sym, h):
    # from 2^28 bytes on a lane reads four rows of 16-bit results: as in pieces, where it reads one
    row = d // 2 + (2 if sym else 4) * (d // g)
    t = (1 << 28) // (h * (4 * d + 2 * row)) + 77
    announce(f"kv4 read of {t} tokens d={d} g={g} h={h}")
    gen = torch.Generator(device="cuda").manual_seed(d)
    n_pages = 40
    k = torch.randn(n_pages * 64, h, d, generator=gen, device="cuda").to(torch.bfloat16)
    v = torch.randn(n_pages * 64, h, d, generator=gen, device="cuda").to(torch.bfloat16)
    cache = B.gq_kv4_empty(n_pages, h, d, 64, g, sym)
    B.gq_kv4_write(k, v, cache, torch.arange(n_pages * 64, device="cuda"), g, sym)
    slots = torch.randint(0, n_pages * 64, (t,), generator=gen, device="cuda")
    slots[9], slots[t - 2] = -1, n_pages * 64
    for odt in (torch.bfloat16, torch.float16):
        ko, vo = B.gq_kv4_read(cache, slots, d, g, sym, odt)
        for a in range(0, t, 4000):
            kw, vw = B.gq_kv4_read(cache, slots[a:a + 4000], d, g, sym, odt)
            assert torch.equal(ko[a:a + 4000], kw) and torch.equal(vo[a:a + 4000], vw)
