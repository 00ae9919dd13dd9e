"""The 4-bit key/value cache where its kernels change shape: many rows read at
once, single sequences and batches of more than 64, row tiles that end with a
worker's share, fp16 results of few rows, the layer that uses it all."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from gpu_util import announce
from kv4_util import attention64, quantise64
from test_gpu_kv4 import DT, Problem, announce_case, fill_random, rows
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,g,sym,h", [(64, 32, True, 32), (96, 96, False, 24), (128, 32, False, 16),
                                       (256, 128, False, 8)])
def test_many_rows_written_and_read(d, g, sym, h):
    # past the size from which a lane reads several rows; the last ones of a ragged count, some skipped
    t = 65536 // h + 37
    announce(f"kv4 many rows d={d} g={g} h={h} t={t}")
    gen = torch.Generator().manual_seed(d)
    k, v = rows(gen, t, h, d, torch.float16), rows(gen, t, h, d, torch.float16)
    n_pages = t // 64 + 2
    slots = torch.randperm(n_pages * 64, generator=gen)[:t]
    slots[5], slots[t - 1] = -1, n_pages * 64
    cache = B.gq_kv4_empty(n_pages, h, d, 64, g, sym)
    fill_random(cache, gen)
    B.gq_kv4_write(k.cuda(), v.cuda(), cache, slots.cuda(), g, sym)
    k32, v32 = B.gq_kv4_read(cache, slots.cuda(), d, g, sym, torch.float32)
    for got, x in ((k32, k), (v32, v)):
        want, _, _ = quantise64(x, g, sym)
        want[[5, t - 1]] = 0.0
        assert torch.equal(got.cpu().double(), want)
    for odt in (torch.bfloat16, torch.float16):
        ko, vo = B.gq_kv4_read(cache, slots.cuda(), d, g, sym, odt)
        assert torch.equal(ko, k32.to(odt)) and torch.equal(vo, v32.to(odt))


@pytest.mark.parametrize("q,kv,h,r", [([1], [5000], 2, 4), ([1], [1025], 1, 1), ([3], [40000], 1, 2),
                                      ([6], [2000], 3, 5)])
def test_one_long_sequence(q, kv, h, r):
    p = Problem(41 + q[0], 128, 64, False, 16, "bf16", h, r, q, kv)
    announce_case(p, "one sequence")
    p.check(*p.run(), what="one sequence")


@pytest.mark.parametrize("q,kv,h,r,d,g", [([300], [300], 2, 1, 128, 128), ([2100], [2100], 1, 8, 64, 32),
                                          ([65], [70], 2, 4, 96, 32), ([200], [900], 1, 2, 256, 32)])
def test_one_prompt(q, kv, h, r, d, g):
    # [2100] with 8 heads: more row tiles than lanes of a wave
    p = Problem(51 + d, d, g, False, 32, "bf16", h, r, q, kv)
    announce_case(p, "one prompt")
    p.check(*p.run(), fp16_operands=True, what="one prompt")


def test_long_prompt_beside_a_short_one():
    # more row tiles than 8 per sequence: the lengths are scanned sequence by sequence
    p = Problem(57, 64, 64, False, 32, "bf16", 2, 4, [1200, 30, 0], [1300, 30, 7])
    announce_case(p, "long prompt beside a short one")
    p.check(*p.run(), fp16_operands=True, what="long prompt beside a short one")
    p = Problem(58, 64, 32, True, 16, "f16", 1, 8, [2, 1100], [90, 1100])
    announce_case(p, "short prompt before a long one")
    p.check(*p.run(window=300), window=300, fp16_operands=True, what="short prompt before a long one")


@pytest.mark.parametrize("max_q", [1, 40])
def test_more_sequences_than_lanes(max_q):
    gen = torch.Generator().manual_seed(3)
    n = 150
    kv = [int(x) for x in torch.randint(0, 200, (n,), generator=gen)]
    kv[70], kv[149] = 1500, 1300
    q = [min(x, int(m)) for x, m in zip(kv, torch.randint(0, max_q + 1, (n,), generator=gen))]
    if max_q == 1:
        q = [1] * n
    p = Problem(61, 64, 64, True, 16, "f16", 2, 2, q, kv)
    announce_case(p, "many sequences")
    a = p.run()
    p.check(*a, fp16_operands=True, what="many sequences")
    b = p.run(max_q_len=1)                      # the other way to share the scan of the lengths
    p.check(*b, fp16_operands=True, what="many sequences, loose bound")


def test_long_and_empty_row_tiles_together():
    # shares that end inside, at and just after a row tile; queries before all keys
    p = Problem(71, 128, 128, False, 16, "bf16", 1, 4, [1] * 20, [0, 3000, 0, 0, 1, 128, 256, 257, 4000, 0] * 2)
    announce_case(p, "empty among long")
    p.check(*p.run(), what="empty among long")
    p = Problem(72, 128, 64, False, 16, "f16", 2, 4, [70, 90, 64, 200], [10, 90, 0, 1200])
    p.check(*p.run(), fp16_operands=True, what="queries before all keys")


@pytest.mark.parametrize("q", [1, 40])
def test_tables_far_wider_than_the_lengths(q):
    # 2^30 positions in a row of the table: more tiles than 32 bits count at the
    # usual grain of the split, so the grain is coarser
    gen = torch.Generator().manual_seed(5)
    kv = [int(x) for x in torch.randint(41, 3000, (32,), generator=gen)]
    kv[3], kv[9], kv[20] = 2900, 41, 512
    p = Problem(91, 64, 64, False, 1024, "bf16", 8, 1, [q] * 32, kv)
    announce_case(p, "wide table")
    table = torch.full((32, 1 << 20), 0x7FFFFFF0, dtype=torch.int32)
    table[:, :p.table.shape[1]] = p.table
    p.check(*p.run(table=table), fp16_operands=True, what="wide table")


@pytest.mark.parametrize("d,g,sym", [(64, 64, True), (128, 32, False), (256, 256, False)])
def test_fp16_result_of_few_rows_is_rounded_once(d, g, sym):
    # Up to 8 rows: what rounding the weights leaves is carried along.  Besides the
    # result's own rounding (half a step, 2^-11, of it) this remains, of the mean
    # |value|: weights in two fp16 parts, 2^-21; exp2 and sums, 2^-20; the scores'
    # (d + 16) 2^-24 of 30 scales and |q|, twice (numerator and denominator), small
    # because the queries are.  One rounding of the weights would be 2^-11.
    for r, q in ((4, [1, 1, 1]), (1, [4, 2, 2]), (8, [1, 1, 1])):
        p = Problem(81 + r, d, g, sym, 16, "f16", 2, r, q, [5, 3, 2], q_scale=2.0 ** -10)
        announce_case(p, "few rows in fp16")
        out, _ = p.run()
        qa = ka = 0
        for n, kv in zip(p.q_lens, p.kv_lens):
            qb, k, v = p.q[qa:qa + n].double(), p.k[ka:ka + kv], p.v[ka:ka + kv]
            want, _, w = attention64(qb, k, v, n, kv, True, 0, d ** -0.5)
            mean = torch.einsum("nhk,khd->nhd", w, v.repeat_interleave(r, 1).abs())
            s_err = d ** -0.5 * (d + 16) * 2.0 ** -24 * 30 * qb.abs().sum(-1) * p.sk[ka:ka + kv].max()
            rest = mean * (2.0 ** -21 + 2.0 ** -20 + 2 * s_err[..., None])
            tol = rest + 2.0 ** -11 * (want.abs() + rest) + 2.0 ** -25
            assert float(s_err.max()) < 2.0 ** -15               # the bound says something
            assert ((out[qa:qa + n].cpu().double() - want).abs() <= tol).all()
            qa, ka = qa + n, ka + kv


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_layer_example(dtype):
    # INT4 projections, cache, attention, graph replays.  Of independent roundings
    # of the 16-bit type (half a step each, relative) the result sees three in
    # sequence: the weights of the attention, its output, the projection's output.
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    announce(f"kv4 layer example {dtype}")
    worst = mod.run((150, 33, 1, 17), 4, hidden=512, q_heads=8, kv_heads=2, head_dim=64, group=64, page=16,
                    n_pages=64, dtype=DT[dtype])
    announce(f"layer: {worst:.2e}")
    assert worst <= 3 * torch.finfo(DT[dtype]).eps / 2
