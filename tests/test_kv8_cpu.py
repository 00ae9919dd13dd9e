"""The 8-bit key/value cache without a GPU: exports, sizes, refusals before any
device call, and the definitions of the tests against themselves."""
import ctypes
import os

import pytest
import torch

import kv8_util as U
from conftest import ROOT
from test_abi import header_functions
from w4a16_dequant_gemm_group_amd import binding as B

FAKE, MIS = 4096, 4096 + 8
BAD, MISALIGNED, UNSUPPORTED = B.GQ_ERR_INVALID_ARG, B.GQ_ERR_MISALIGNED, B.GQ_ERR_UNSUPPORTED


def layout(**kw):
    a = dict(kv_heads=8, head_dim=128, page_size=64)
    a.update(kw)
    return B.GqKv8Layout(**a)


def make(cls, base, kw):
    a = {**base, **kw}
    return ctypes.byref(cls(*(a[f] for f, _ in cls._fields_)))


def append_args(**kw):
    return make(B.GqKv8AppendArgs, dict(
        k=FAKE, k_token_stride=1024, k_head_stride=128, v=FAKE, v_token_stride=1024, v_head_stride=128,
        dtype=B.GQ_BF16, tokens=3, cache=FAKE, n_pages=100, layout=layout(), page_table=FAKE, batch=3,
        table_pages=40, kv_lens=FAKE, starts=None, bounds=None), kw)


def attn_args(**kw):
    return make(B.GqKv8AttentionArgs, dict(
        q=FAKE, q_token_stride=4096, q_head_stride=128, q_tokens=2, q_heads=32, dtype=B.GQ_BF16, cache=FAKE,
        n_pages=100, layout=layout(), page_table=FAKE, batch=2, table_pages=40, head_tables=0, kv_lens=FAKE,
        q_starts=None, max_q_len=1, max_kv_len=2560, causal=1, window=0, scale=0.1, out=FAKE, lse=None), kw)


def select_args(**kw):
    return make(B.GqKv8SelectArgs, dict(
        q=FAKE, q_token_stride=4096, q_head_stride=128, q_tokens=2, q_heads=32, dtype=B.GQ_BF16, bounds=FAKE,
        n_pages=100, layout=layout(), page_table=FAKE, batch=2, table_pages=40, kv_lens=FAKE, q_starts=None,
        max_kv_len=2560, keep=8, first=1, last=1, pages=FAKE, lens=FAKE), kw)


def test_exports_every_declared_symbol():
    names = header_functions(os.path.join(ROOT, "include", "gq_kv8.h"))
    assert set(names) == set(B.KV8_EXPORTS) and len(names) == 7
    for n in names:
        assert hasattr(B.lib(), n), n


@pytest.mark.parametrize("d,h,page", [(128, 8, 64), (96, 1, 16), (64, 3, 1024), (256, 2, 32)])
def test_cache_bytes(d, h, page):
    n = ctypes.c_size_t()
    assert B.lib().gq_kv8_cache_bytes(7, layout(head_dim=d, kv_heads=h, page_size=page), ctypes.byref(n)) == B.GQ_OK
    assert n.value == 7 * h * page * 2 * d + 7 * h * (page // 16) * 8
    c = B.gq_kv8_empty(7, h, d, page, device="cpu")
    assert c.numel() == n.value and c.dtype == torch.uint8
    assert B.gq_kv8_bounds_empty(7, h, d, torch.float16, device="cpu").shape == (7, h, 2, d)


@pytest.mark.parametrize("kw,expect", [
    (dict(kv_heads=0), BAD), (dict(kv_heads=65536), BAD), (dict(head_dim=80), BAD), (dict(head_dim=0), BAD),
    (dict(head_dim=192), UNSUPPORTED), (dict(head_dim=32), UNSUPPORTED), (dict(page_size=48), BAD),
    (dict(page_size=8), BAD), (dict(page_size=2048), BAD),
])
def test_layout_refusals(kw, expect):
    L, lay, n = B.lib(), layout(**kw), ctypes.c_size_t()
    heads = dict(q_heads=max(1, kw.get("kv_heads", 8)))
    assert L.gq_kv8_cache_bytes(4, lay, ctypes.byref(n)) == expect
    assert L.gq_kv8_append(append_args(layout=lay), None) == expect
    assert L.gq_kv8_read(FAKE, 4, lay, FAKE, 3, FAKE, FAKE, B.GQ_F32, None) == expect
    assert L.gq_kv8_attention(attn_args(layout=lay, **heads), FAKE, 1 << 40, None) == expect
    assert L.gq_kv8_select(select_args(layout=lay, **heads), FAKE, 1 << 40, None) == expect


def test_cache_limits():
    L, n = B.lib(), ctypes.c_size_t()
    for pages in (0, -1, 1 << 31):
        assert L.gq_kv8_cache_bytes(pages, layout(), ctypes.byref(n)) == BAD
    big = layout(kv_heads=65535, head_dim=256, page_size=1024)
    assert L.gq_kv8_cache_bytes((1 << 31) - 1, big, ctypes.byref(n)) == BAD
    assert L.gq_kv8_cache_bytes(1 << 27, big, ctypes.byref(n)) == BAD        # 2^62 and 0.1 %
    assert L.gq_kv8_cache_bytes(1 << 26, big, ctypes.byref(n)) == B.GQ_OK and n.value == (1 << 26) * 65535 * 64 * 8200
    assert L.gq_kv8_cache_bytes(4, layout(), None) == BAD


def test_append_refusals():
    f = lambda **kw: B.lib().gq_kv8_append(append_args(**kw), None)
    for kw in (dict(k=None), dict(v=None), dict(cache=None), dict(kv_lens=None), dict(page_table=None), dict(n_pages=0),
               dict(tokens=-1), dict(tokens=2), dict(tokens=(1 << 30) + 1), dict(batch=-1), dict(batch=(1 << 24) + 1),
               dict(table_pages=-1), dict(table_pages=1 << 25), dict(dtype=7), dict(k_token_stride=1 << 41),
               dict(v_head_stride=-(1 << 41))):
        assert f(**kw) == BAD, kw
    assert f(dtype=B.GQ_F32) == UNSUPPORTED
    for kw in (dict(k=MIS), dict(v=MIS), dict(cache=MIS), dict(bounds=MIS), dict(k_token_stride=1028),
               dict(v_head_stride=4), dict(page_table=FAKE + 2), dict(kv_lens=FAKE + 2), dict(starts=FAKE + 2)):
        assert f(**kw) == MISALIGNED, kw
    assert B.lib().gq_kv8_append(None, None) == BAD
    assert f(tokens=0, k=None) == B.GQ_OK and f(batch=0, k=None) == B.GQ_OK


def test_read_refusals():
    r = lambda k=FAKE, v=FAKE, dt=B.GQ_BF16, t=3, s=FAKE, c=FAKE, n=4: \
        B.lib().gq_kv8_read(c, n, layout(), s, t, k, v, dt, None)
    for kw in (dict(k=None), dict(v=None), dict(s=None), dict(c=None), dict(t=-1), dict(t=(1 << 30) + 1), dict(n=0), dict(dt=5)):
        assert r(**kw) == BAD, kw
    for kw in (dict(k=MIS), dict(v=MIS), dict(c=MIS), dict(s=FAKE + 4)):
        assert r(**kw) == MISALIGNED, kw
    assert r(t=0, k=None) == B.GQ_OK


def test_attention_refusals():
    L = B.lib()
    f = lambda ws=FAKE, n=1 << 40, **kw: L.gq_kv8_attention(attn_args(**kw), ws, n, None)
    for kw in (dict(q=None), dict(cache=None), dict(out=None), dict(kv_lens=None), dict(page_table=None),
               dict(n_pages=0), dict(q_heads=0), dict(q_heads=33), dict(q_heads=8 * 65), dict(dtype=9),
               dict(q_tokens=-1), dict(q_tokens=1), dict(batch=-1), dict(table_pages=-1), dict(head_tables=2),
               dict(max_q_len=-1), dict(max_kv_len=-1), dict(max_kv_len=(1 << 30) + 1), dict(causal=2), dict(window=-1),
               dict(causal=0, window=5), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(q_tokens=1 << 30), dict(table_pages=1 << 30)):
        assert f(**kw) == BAD, kw
    assert f(dtype=B.GQ_F32) == UNSUPPORTED
    for kw in (dict(q=MIS), dict(cache=MIS), dict(out=MIS), dict(q_token_stride=4100), dict(q_head_stride=4),
               dict(lse=FAKE + 2), dict(kv_lens=FAKE + 2), dict(page_table=FAKE + 2), dict(q_starts=FAKE + 2)):
        assert f(**kw) == MISALIGNED, kw
    need = ctypes.c_size_t()
    assert L.gq_kv8_attention_workspace_size(attn_args(), ctypes.byref(need)) == B.GQ_OK and need.value > 0
    assert f(ws=None) == BAD and f(n=need.value - 1) == BAD and f(ws=MIS) == MISALIGNED
    assert L.gq_kv8_attention(None, FAKE, 1 << 40, None) == BAD
    assert L.gq_kv8_attention_workspace_size(attn_args(), None) == BAD
    assert f(batch=0, q_tokens=0, q=None, ws=None) == B.GQ_OK
    assert f(q_tokens=0, q_starts=FAKE, ws=None) == B.GQ_OK


def test_select_refusals():
    L = B.lib()
    f = lambda ws=FAKE, n=1 << 40, **kw: L.gq_kv8_select(select_args(**kw), ws, n, None)
    for kw in (dict(q=None), dict(bounds=None), dict(pages=None), dict(lens=None), dict(kv_lens=None),
               dict(page_table=None), dict(n_pages=0), dict(q_heads=0), dict(q_heads=33), dict(q_heads=8 * 65),
               dict(dtype=9), dict(q_tokens=-1), dict(q_tokens=1), dict(batch=-1), dict(max_kv_len=-1),
               dict(keep=0), dict(keep=65537), dict(keep=1), dict(first=-1), dict(last=0), dict(first=5, last=4),
               dict(first=(1 << 31) - 1, last=(1 << 31) - 1)):
        assert f(**kw) == BAD, kw
    assert f(dtype=B.GQ_F32) == UNSUPPORTED
    for kw in (dict(q=MIS), dict(bounds=MIS), dict(q_token_stride=4100), dict(pages=FAKE + 2), dict(lens=FAKE + 2),
               dict(kv_lens=FAKE + 2), dict(page_table=FAKE + 2), dict(q_starts=FAKE + 2)):
        assert f(**kw) == MISALIGNED, kw
    need = ctypes.c_size_t()
    assert L.gq_kv8_select_workspace_size(select_args(), ctypes.byref(need)) == B.GQ_OK
    assert need.value == 2 * 8 * 40 * 8
    assert f(ws=None) == BAD and f(n=need.value - 1) == BAD and f(ws=MIS) == MISALIGNED
    assert L.gq_kv8_select(None, FAKE, 1 << 40, None) == BAD
    assert L.gq_kv8_select_workspace_size(select_args(), None) == BAD
    assert f(q_tokens=0, q_starts=FAKE, q=None, ws=None) == B.GQ_OK


def test_binding_checks():
    bf = torch.bfloat16
    k, cache = torch.zeros(2, 4, 64, dtype=bf), B.gq_kv8_empty(6, 4, 64, 16, device="cpu")
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    bounds = B.gq_kv8_bounds_empty(6, 4, 64, device="cpu")
    for a, exc in [((k.float(), k, cache, table, lens), TypeError), ((k, k.half(), cache, table, lens), TypeError),
                   ((k, k[:1], cache, table, lens), ValueError), ((k[:, :2], k[:, :2], cache, table, lens), ValueError),
                   ((k, k, cache[..., :-8], table, lens), ValueError), ((k, k, cache, table[0], lens), ValueError),
                   ((k, k, cache, table.long(), lens), TypeError), ((k, k, cache, table, lens[:1]), ValueError),
                   ((k[:1], k[:1], cache, table, lens), ValueError), ((k, k, cache, table, lens, lens), ValueError),
                   ((k, k, cache, table, lens, None, bounds.half()), TypeError),
                   ((k, k, cache, table, lens, None, bounds[:3]), ValueError),
                   ((k, k, cache, table, lens, None, bounds), ValueError)]:     # the last: not on a GPU
        with pytest.raises(exc):
            B.gq_kv8_append(*a)
    q = torch.zeros(2, 8, 64, dtype=bf)
    for a, kw, exc in [((q.float(), cache, table, lens), {}, TypeError), ((q[:, :6], cache, table, lens), {}, ValueError),
                       ((q, cache, table[:, None].expand(2, 2, 3).contiguous(), lens), {}, ValueError),
                       ((q[:1], cache, table, lens), {}, ValueError), ((q, cache, table, lens), dict(q_starts=lens), ValueError),
                       ((q, cache, table, lens), dict(out=q.half()), TypeError),
                       ((q, cache, table, lens), dict(lse=torch.zeros(2, 4)), ValueError),
                       ((q, cache, table, lens), {}, ValueError)]:
        with pytest.raises(exc):
            B.gq_kv8_attention(*a, **kw)
    for a, kw, exc in [((q.half(), bounds, table, lens, 4), {}, TypeError), ((q, bounds, table, lens, 4, 24), {}, ValueError),
                       ((q[:, :6], bounds, table, lens, 4), {}, ValueError), ((q, bounds, table, lens, 1), {}, ValueError),
                       ((q, bounds, table, lens, 4), dict(last=0), ValueError),
                       ((q, bounds, table, lens, 4), dict(pages=torch.zeros(2, 4, 5, dtype=torch.int32)), ValueError),
                       ((q, bounds, table, lens, 4), {}, ValueError)]:
        with pytest.raises(exc):
            B.gq_kv8_select(*a, **kw)
    with pytest.raises(ValueError):
        B.gq_kv8_read(cache, torch.zeros(3, 1, dtype=torch.int64), 64)
    with pytest.raises(ValueError):
        B.gq_kv8_empty(3, 4, 80, device="cpu")
    with pytest.raises(ValueError):
        B.gq_kv8_empty(3, 4, 64, 24, device="cpu")
    with pytest.raises(TypeError):
        B.gq_kv8_bounds_empty(3, 4, 64, torch.float32, device="cpu")


def test_definition_of_blocks():
    # a block filled in two calls: the scale only grows, older codes are rounded again
    b = U.Blocks(2).append(torch.tensor([[1.27, -0.635], [0.0, 0.004]]))
    assert b.scales == [float(torch.tensor(1.27, dtype=torch.float32).double().div(127).float())]
    assert b.codes.tolist() == [[127, -64], [0, 0]]       # 63.5 rounds to even
    b.append(torch.tensor([[2.54, 0.0]]))
    assert b.codes.tolist() == [[64, -32], [0, 0], [127, 0]]
    b.append(torch.tensor([[0.02, 0.0]]))
    assert b.codes.tolist()[3] == [1, 0]
    # blocks begin at multiples of 16, and zeros have the least scale
    z = U.Blocks(1).append(torch.zeros(17, 1))
    assert z.scales == [U.LEAST, U.LEAST] and z.codes.shape == (17, 1)


@pytest.mark.parametrize("args,pack", [
    (B.GqRopeArgs, B._rope_args), (B.GqKv8AppendArgs, B._kv8_append_args),
    (B.GqKv8AttentionArgs, B._kv8_attention_args), (B.GqKv8SelectArgs, B._kv8_select_args)])
def test_packed_arguments_are_the_structure(args, pack):
    """Every field in its place; a value that does not fit its field is refused, not cut."""
    flat, whole, n = [], [], 0
    for _, t in args._fields_:
        if t is B.GqKv8Layout:
            flat += [n + 1, n + 2, n + 3]
            whole.append(B.GqKv8Layout(n + 1, n + 2, n + 3))
            n += 3
        else:
            n += 1
            v = n + 0.5 if t is ctypes.c_float else n
            flat.append(v)
            whole.append(v)
    assert pack(*flat) == bytes(args(*whole))
    for i, v in enumerate(flat):
        # (a float beyond fp32 becomes infinity, which the library refuses)
        for bad in (None, "x") if isinstance(v, float) else (None, "x", 1.5, 1 << 70, -(1 << 70)):
            with pytest.raises(ValueError):
                pack(*flat[:i], bad, *flat[i + 1:])
