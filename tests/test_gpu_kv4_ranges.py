"""Attention over the 4-bit cache at the ends of its number ranges: large and
small queries and scales, a key that takes nearly all the weight, rows of zeros,
neighbours of very different size."""
import math

import pytest
import torch

from gpu_util import announce
from kv4_bounds import exact_key_bounds
from kv4_util import attention64, quantise64
from test_gpu_kv4 import DT, rows
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu


def attend(q, k, v, g, sym=False, scale=None, copies=1):
    """One sequence, q [n, HQ, D] over a cache of k, v [kv, H, D]: out and lse, the
    definition's, and the bounds of both.  copies: so many sequences of the same
    queries and pages, enough of them that a workgroup walks over all keys of one."""
    n, kv, h, d = q.shape[0], k.shape[0], k.shape[1], k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    page, n_pages = 64, -(-kv // 64)
    cache = B.gq_kv4_empty(n_pages, h, d, page, g, sym)
    cache.fill_(0xFF)
    B.gq_kv4_write(k.cuda(), v.cuda(), cache, torch.arange(kv, device="cuda"), g, sym)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").repeat(copies, 1)
    out, lse = B.gq_kv4_attention(q.cuda().repeat(copies, 1, 1), cache, table,
                                  torch.full((copies,), kv, dtype=torch.int32, device="cuda"), g, sym,
                                  q_starts=torch.arange(0, n * copies + 1, n, dtype=torch.int32, device="cuda"),
                                  max_q_len=n, max_kv_len=kv, scale=scale, return_lse=True)
    out, lse = out.view(copies, n, -1, d), lse.view(copies, n, -1)
    k64, sk, _ = quantise64(k, g, sym)
    v64, sv, _ = quantise64(v, g, sym)
    sv = sv * (v64.unflatten(-1, (d // g, g)) != 0).any(-1)
    q64 = q.double()
    o, l, p = attention64(q64, k64, v64, n, kv, True, 0, scale)
    rows = n * (q.shape[1] // h)
    kind = "many" if rows > 32 else "once" if rows <= 8 and q.dtype == torch.float16 else "few"
    tol, ltol = exact_key_bounds(q64, k64, v64, sk.amax(-1), sv.amax(-1), o, l, p, scale, q.dtype, kind)
    return out.cpu().double(), lse.cpu().double(), o, l, tol, ltol


def check(what, out, lse, o, l, tol, ltol):
    assert torch.isfinite(out).all() and torch.isfinite(lse).all(), what
    worst, worst_l = float(((out - o).abs() / tol).max()), float(((lse - l).abs() / ltol).max())
    announce(f"{what}: error / bound {worst:.3f}, lse {worst_l:.3f}")
    assert worst <= 1.0 and worst_l <= 1.0, what


FORMS = [(128, 128, False), (128, 32, False), (256, 64, False), (64, 32, True)]


@pytest.mark.parametrize("n", [2, 70])
@pytest.mark.parametrize("d,g,sym", FORMS)
def test_large_queries(d, g, sym, n):
    # queries up to bf16's largest, keys so small that the scores are ordinary
    gen = torch.Generator().manual_seed(d + g)
    for e in (90, 101, 102, 115, 127):
        q = torch.randn(n, 2, d, generator=gen)
        q[0, 0, 3], q[n - 1, 1, 5] = 1.9, -1.8
        q = (q.clamp(-1.9, 1.9) * 2.0 ** e).to(torch.bfloat16)
        k = (rows(gen, 200, 1, d, torch.bfloat16).double() * 2.0 ** -12).to(torch.bfloat16)
        v = rows(gen, 200, 1, d, torch.bfloat16)
        check(f"queries to 2^{e}", *attend(q, k, v, g, sym, scale=d ** -0.5 * 2.0 ** (11 - e)))


@pytest.mark.parametrize("n", [2, 70])
@pytest.mark.parametrize("d,g,sym", FORMS)
def test_small_queries(d, g, sym, n):
    # queries down to bf16's smallest normal ones, a scale that makes up for it
    gen = torch.Generator().manual_seed(11 * d + g)
    for e in (-59, -64, -100, -124):
        q = (torch.randn(n, 2, d, generator=gen) * 2.0 ** e).to(torch.bfloat16)
        k, v = rows(gen, 200, 1, d, torch.bfloat16), rows(gen, 200, 1, d, torch.bfloat16)
        check(f"queries of 2^{e}", *attend(q, k, v, g, sym, scale=d ** -0.5 * 2.0 ** -e))


@pytest.mark.parametrize("n", [2, 70])
@pytest.mark.parametrize("d,g,sym", FORMS)
def test_tiny_scale(d, g, sym, n):
    # scores that vanish in fp32: the mean of the keys that a row sees, no more of them
    gen = torch.Generator().manual_seed(9 * d + g)
    q = 1e-3 * torch.randn(n, 2, d, generator=gen)
    k, v = rows(gen, 200, 1, d, torch.bfloat16), rows(gen, 200, 1, d, torch.bfloat16)
    for scale in (1e-12, 1e-30, 1e-38):
        check(f"scale {scale}", *attend(q.to(torch.bfloat16), k, v, g, sym, scale=scale))
        check(f"scale {scale}, no query", *attend(torch.zeros_like(q).to(torch.bfloat16), k, v, g, sym, scale=scale))


def with_sink(gen, kv, d, dtype, ahead, spread=0.3):
    """Queries and keys such that key 0's score is `ahead` nats above the others'."""
    u = torch.randn(d, generator=gen)
    u = u / u.norm()
    k = spread * torch.randn(kv, 1, d, generator=gen)
    k -= (k @ u)[..., None] * u
    k[0, 0] = 4.0 * u
    make_q = lambda n, hq: (torch.randn(n, hq, d, generator=gen) * 0.5 + ahead / 4.0 * d ** 0.5 * u).to(dtype)
    return make_q, k.to(dtype)


@pytest.mark.parametrize("n,dtype", [(1, "f16"), (2, "bf16"), (9, "f16"), (70, "bf16"), (70, "f16")])
@pytest.mark.parametrize("d,g,sym", FORMS)
def test_a_key_that_takes_nearly_all_the_weight(d, g, sym, n, dtype):
    # an attention sink: its value is small (in one group of channels at least, where
    # there are several), so the result is what the many light keys add up to
    gen = torch.Generator().manual_seed(3 * d + g)
    for kv, ahead in ((4096, 16.0), (4096, 18.0), (9000, 19.0)):
        make_q, k = with_sink(gen, kv, d, DT[dtype], ahead)
        v = (rows(gen, kv, 1, d, torch.float32).abs() * 0.5).to(DT[dtype])
        v[0] = 1e-5
        if g < d:
            v[0, 0, :g] = torch.rand(g, generator=gen) * 4.0
        check(f"sink {ahead} ahead of {kv} keys", *attend(make_q(n, 2), k, v, g, sym, copies=300))


@pytest.mark.parametrize("n,dtype", [(1, "f16"), (2, "bf16"), (9, "bf16"), (70, "bf16"), (70, "f16")])
@pytest.mark.parametrize("d,g,sym", FORMS)
def test_rows_of_zeros_beside_small_values(d, g, sym, n, dtype):
    # a zero row stands for zeros whatever its scale is: it must not set the range
    gen = torch.Generator().manual_seed(5 * d + g)
    for ahead, small in ((12.0, 1e-3), (14.0, 0.02), (18.0, 1e-4)):
        make_q, k = with_sink(gen, 3000, d, DT[dtype], ahead)
        v = (rows(gen, 3000, 1, d, torch.float32).abs() * small).to(DT[dtype])
        v[0] = 0.0
        v[700:720] = 0.0
        check(f"zero row {ahead} ahead of values of {small}", *attend(make_q(n, 2), k, v, g, sym, copies=300))


@pytest.mark.parametrize("n,dtype", [(2, "bf16"), (70, "bf16"), (70, "f16")])
@pytest.mark.parametrize("d,g,sym", FORMS)
def test_neighbours_of_very_different_size(d, g, sym, n, dtype):
    # key 21 and its value are 2^19 times those of the tokens around them, but no
    # query gives it weight: the others lose nothing by standing next to it
    gen = torch.Generator().manual_seed(7 * d + g)
    kv = 96
    q = 1.5 * torch.randn(n, 2, d, generator=gen)
    q[..., 0] = -1.0
    k, v = 2.0 ** -6 * rows(gen, kv, 1, d, torch.float32), 2.0 ** -8 * rows(gen, kv, 1, d, torch.float32)
    k[..., 0] = 0.0
    k[21] = 0.0
    k[21, 0, 0], k[21, 0, 1] = 2.0 ** 15, 2.0 ** -12
    v[21] = 2.0 ** 14 * torch.rand(1, d, generator=gen)
    check("neighbours of different size", *attend(q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), g, sym))


@pytest.mark.parametrize("n", [2, 70])
@pytest.mark.parametrize("d,g,sym", FORMS)
def test_nonfinite_queries_that_see_no_key(d, g, sym, n):
    # pages that do not exist, whole or from some page on; keys after a query's position
    announce(f"kv4 non-finite queries without keys d={d} g={g} n={n}")
    gen = torch.Generator().manual_seed(d)
    cache = B.gq_kv4_empty(8, 1, d, 16, g, sym)
    k = rows(gen, 128, 1, d, torch.bfloat16).cuda()
    B.gq_kv4_write(k, k, cache, torch.arange(128, device="cuda"), g, sym)
    q = torch.randn(3 * n, 2, d, generator=gen).to(torch.bfloat16)
    q[:, 0, 3], q[:, 1, 5] = math.nan, -math.inf
    table = torch.tensor([[-1] * 8, [8, -5, 1 << 30, 9, -1, -1, -1, -1], list(range(8))], dtype=torch.int32)
    lens = torch.tensor([128, 77, 0], dtype=torch.int32)
    out, lse = B.gq_kv4_attention(q.cuda(), cache, table.cuda(), lens.cuda(), g, sym,
                                  q_starts=torch.tensor([0, n, 2 * n, 3 * n], dtype=torch.int32).cuda(), max_q_len=n,
                                  max_kv_len=128, causal=False, return_lse=True)
    assert not out.any() and (lse == -math.inf).all()
