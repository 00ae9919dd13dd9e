"""The 4-bit key/value cache without a GPU: the header's entry points are
exported and bound, and wrong calls are refused before any device call."""
import ctypes
import os

import pytest
import torch

from conftest import ROOT
from test_abi import header_functions
from w4a16_dequant_gemm_group_amd import binding as B

FAKE = ctypes.c_void_p(4096)
MIS = ctypes.c_void_p(4096 + 8)


def layout(**kw):
    a = dict(kv_heads=8, head_dim=128, page_size=64, group_size=128, symmetric=0)
    a.update(kw)
    return B.GqKv4Layout(**a)


def test_exports_every_declared_symbol():
    names = header_functions(os.path.join(ROOT, "include", "gq_kv.h"))
    assert set(names) == set(B.KV_EXPORTS) and len(names) == 5
    for n in names:
        assert hasattr(B.lib(), n), n


@pytest.mark.parametrize("d,g,sym,page", [(128, 128, 0, 64), (128, 32, 0, 16), (96, 96, 1, 128),
                                          (64, 32, 1, 32), (256, 64, 0, 1024)])
def test_cache_bytes(d, g, sym, page):
    n = ctypes.c_size_t()
    assert B.lib().gq_kv4_cache_bytes(7, layout(head_dim=d, group_size=g, symmetric=sym, page_size=page),
                                      ctypes.byref(n)) == B.GQ_OK
    row = d // 2 + (2 if sym else 4) * (d // g)
    assert n.value == 7 * page * 8 * 2 * row
    c = B.gq_kv4_empty(7, 8, d, page, g, bool(sym), device="cpu")
    assert c.numel() == n.value and c.dtype == torch.uint8


@pytest.mark.parametrize("kw,expect", [
    (dict(kv_heads=0), B.GQ_ERR_INVALID_ARG), (dict(kv_heads=65536), B.GQ_ERR_INVALID_ARG),
    (dict(head_dim=80, group_size=80), B.GQ_ERR_INVALID_ARG),
    (dict(head_dim=192, group_size=64), B.GQ_ERR_UNSUPPORTED),
    (dict(page_size=48), B.GQ_ERR_INVALID_ARG), (dict(page_size=8), B.GQ_ERR_INVALID_ARG),
    (dict(page_size=2048), B.GQ_ERR_INVALID_ARG),
    (dict(group_size=48), B.GQ_ERR_INVALID_ARG), (dict(group_size=96), B.GQ_ERR_INVALID_ARG),
    (dict(group_size=0), B.GQ_ERR_INVALID_ARG), (dict(symmetric=2), B.GQ_ERR_INVALID_ARG),
])
def test_layout_refusals(kw, expect):
    L, lay, n = B.lib(), layout(**kw), ctypes.c_size_t()
    assert L.gq_kv4_cache_bytes(4, lay, ctypes.byref(n)) == expect
    assert L.gq_kv4_write(FAKE, 1024, 128, FAKE, 1024, 128, B.GQ_BF16, 3, FAKE, FAKE, 4, lay, None) == expect
    assert L.gq_kv4_read(FAKE, 4, lay, FAKE, 3, FAKE, FAKE, B.GQ_F32, None) == expect
    a = attn_args(layout=lay)
    assert L.gq_kv4_attention(ctypes.byref(a), FAKE, 1 << 30, None) == expect


def test_store_refusals():
    L, lay = B.lib(), layout()
    w = lambda k=FAKE, kts=1024, khs=128, v=FAKE, vts=1024, vhs=128, dt=B.GQ_BF16, t=3, s=FAKE, c=FAKE, n=4: \
        L.gq_kv4_write(k, kts, khs, v, vts, vhs, dt, t, s, c, n, lay, None)
    for kw in (dict(k=None), dict(v=None), dict(s=None), dict(c=None), dict(t=-1), dict(n=0),
               dict(n=1 << 31), dict(dt=7), dict(kts=1 << 41)):
        assert w(**kw) == B.GQ_ERR_INVALID_ARG, kw
    assert w(dt=B.GQ_F32) == B.GQ_ERR_UNSUPPORTED
    for kw in (dict(k=MIS), dict(v=MIS), dict(c=MIS), dict(s=ctypes.c_void_p(4100)), dict(kts=1028),
               dict(vhs=132)):
        assert w(**kw) == B.GQ_ERR_MISALIGNED, kw
    assert w(t=0, k=None) == B.GQ_OK
    r = lambda k=FAKE, v=FAKE, dt=B.GQ_BF16, t=3, s=FAKE, c=FAKE, n=4: \
        L.gq_kv4_read(c, n, lay, s, t, k, v, dt, None)
    for kw in (dict(k=None), dict(v=None), dict(s=None), dict(c=None), dict(t=-1), dict(n=0), dict(dt=5)):
        assert r(**kw) == B.GQ_ERR_INVALID_ARG, kw
    for kw in (dict(k=MIS), dict(v=MIS), dict(c=MIS)):
        assert r(**kw) == B.GQ_ERR_MISALIGNED, kw
    assert r(t=0, k=None) == B.GQ_OK
    assert L.gq_kv4_cache_bytes(4, lay, None) == B.GQ_ERR_INVALID_ARG


def attn_args(**kw):
    a = dict(q=FAKE, q_token_stride=4096, q_head_stride=128, q_tokens=2, q_heads=32, dtype=B.GQ_BF16,
             cache=FAKE, n_pages=100, layout=layout(), page_table=FAKE, batch=2, table_pages=40,
             kv_lens=FAKE, q_starts=None, max_q_len=1, max_kv_len=2560, causal=1, window=0, scale=0.1,
             out=FAKE, lse=None)
    a.update(kw)
    return B.GqKv4AttentionArgs(*(getattr(a[f], "value", a[f]) if f != "layout" else a[f]
                                  for f, _ in B.GqKv4AttentionArgs._fields_))


def test_attention_refusals():
    L = B.lib()

    def call(ws=FAKE, n=1 << 30, **kw):
        return L.gq_kv4_attention(ctypes.byref(attn_args(**kw)), ws, n, None)
    for kw in (dict(q=None), dict(cache=None), dict(out=None), dict(kv_lens=None), dict(page_table=None),
               dict(n_pages=0), dict(q_heads=0), dict(q_heads=33), dict(q_heads=8 * 65), dict(dtype=9),
               dict(q_tokens=-1), dict(q_tokens=1), dict(batch=-1), dict(table_pages=-1),
               dict(max_q_len=-1), dict(max_kv_len=-1), dict(causal=2), dict(window=-1),
               dict(causal=0, window=5), dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(q_tokens=1 << 30), dict(table_pages=1 << 30)):
        assert call(**kw) == B.GQ_ERR_INVALID_ARG, kw
    assert call(dtype=B.GQ_F32) == B.GQ_ERR_UNSUPPORTED
    for kw in (dict(q=MIS), dict(cache=MIS), dict(out=MIS), dict(q_token_stride=4100),
               dict(q_head_stride=4), dict(lse=ctypes.c_void_p(4098)),
               dict(kv_lens=ctypes.c_void_p(4098)), dict(page_table=ctypes.c_void_p(4098)),
               dict(q_starts=ctypes.c_void_p(4098))):
        assert call(**kw) == B.GQ_ERR_MISALIGNED, kw
    need = ctypes.c_size_t()
    assert L.gq_kv4_attention_workspace_size(ctypes.byref(attn_args()), ctypes.byref(need)) == B.GQ_OK
    assert need.value > 0
    assert call(ws=None) == B.GQ_ERR_INVALID_ARG
    assert call(n=need.value - 1) == B.GQ_ERR_INVALID_ARG
    assert call(ws=MIS) == B.GQ_ERR_MISALIGNED
    assert L.gq_kv4_attention(None, FAKE, 1 << 30, None) == B.GQ_ERR_INVALID_ARG
    assert L.gq_kv4_attention_workspace_size(ctypes.byref(attn_args()), None) == B.GQ_ERR_INVALID_ARG
    assert call(batch=0, q_tokens=0, q=None, ws=None) == B.GQ_OK
    assert call(q_tokens=0, q_starts=FAKE, ws=None) == B.GQ_OK


def test_binding_checks_tensors_before_any_call():
    k = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    cache = B.gq_kv4_empty(4, 2, 128, 16, 128, False, device="cpu")
    slots = torch.arange(5)
    for over, exc, msg in [
        (dict(k=k.float()), TypeError, "k: dtype"),
        (dict(v=k.half()), TypeError, "v: dtype"),
        (dict(v=k[:4]), ValueError, "v has 4 tokens"),
        (dict(v=k[:, :1]), ValueError, "v has shape"),
        (dict(k=k[:, :1], v=k[:, :1]), ValueError, "cache has 2 heads"),
        (dict(slots=slots.int()), TypeError, "slots: dtype"),
        (dict(slots=slots[:4]), ValueError, "slots has shape"),
        (dict(g=64), ValueError, "cache has shape"),
        (dict(g=48), ValueError, "group_size"),
        (dict(sym=True), ValueError, "cache has shape"),
        (dict(cache=cache.int()), TypeError, "cache: dtype"),
        (dict(k=torch.zeros(5, 2, 132, dtype=torch.bfloat16)[..., ::2]), ValueError, "k: strides"),
        (dict(k=torch.zeros(5, 2, 129, dtype=torch.bfloat16)[..., :128]), ValueError, "k: strides"),
        (dict(), ValueError, "must be a GPU tensor"),
    ]:
        a = dict(k=k, v=k, cache=cache, slots=slots, g=128, sym=False)
        a.update(over)
        with pytest.raises(exc, match=msg):
            B.gq_kv4_write(a["k"], a["v"], a["cache"], a["slots"], a["g"], a["sym"])
    with pytest.raises(TypeError, match="out_dtype"):
        B.gq_kv4_read(cache, slots, 128, out_dtype=torch.int8)
    with pytest.raises(ValueError, match="head_dim 80"):
        B.gq_kv4_read(cache, slots, 80)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        B.gq_kv4_read(cache, slots, 128)
    for kw in (dict(page_size=24), dict(head_dim=72), dict(group_size=96), dict(n_pages=0)):
        a = dict(n_pages=2, kv_heads=2, head_dim=128, page_size=16, group_size=128, device="cpu")
        a.update(kw)
        with pytest.raises(ValueError):
            B.gq_kv4_empty(**a)
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    table = torch.zeros(3, 2, dtype=torch.int32)
    lens = torch.zeros(3, dtype=torch.int32)
    for over, exc, msg in [
        (dict(q=q.float()), TypeError, "q: dtype"),
        (dict(q=q[:, :3]), ValueError, "not a multiple"),
        (dict(table=table.long()), TypeError, "page_table: dtype"),
        (dict(table=table[0]), ValueError, "page_table must be"),
        (dict(lens=lens[:2]), ValueError, "kv_lens has shape"),
        (dict(q=q[:2]), ValueError, "needs q_starts"),
        (dict(starts=lens), ValueError, "q_starts has shape"),
        (dict(out=torch.zeros(3, 4, 127, dtype=torch.bfloat16)), ValueError, "out has shape"),
        (dict(lse=torch.zeros(3, 3)), ValueError, "lse has shape"),
        (dict(), ValueError, "must be a GPU tensor"),
    ]:
        a = dict(q=q, table=table, lens=lens, starts=None, out=None, lse=None)
        a.update(over)
        with pytest.raises(exc, match=msg):
            B.gq_kv4_attention(a["q"], cache, a["table"], a["lens"], q_starts=a["starts"], out=a["out"],
                               lse=a["lse"])
