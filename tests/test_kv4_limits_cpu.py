"""The 4-bit key/value cache at the ends of what its checks accept, without a GPU."""
import ctypes

import pytest

from test_kv4_cpu import FAKE, attn_args, layout
from w4a16_dequant_gemm_group_amd import binding as B

# 65535 heads x 1024 tokens x 2 x (128 bytes of codes + 8 groups of 4 bytes) is 21 GB a page
WIDE = dict(kv_heads=65535, head_dim=256, group_size=32, page_size=1024)
PAGE = 65535 * 1024 * 2 * (128 + 32)


@pytest.mark.parametrize("pages", [(1 << 63) // PAGE + 1, (1 << 31) - 1])
def test_a_cache_beyond_63_bits_is_refused(pages):
    # its offsets would not fit; the size came back wrapped and small
    L, lay, n = B.lib(), layout(**WIDE), ctypes.c_size_t()
    assert L.gq_kv4_cache_bytes(pages, lay, ctypes.byref(n)) == B.GQ_ERR_INVALID_ARG
    assert n.value == 0
    assert L.gq_kv4_write(FAKE, 65535 * 256, 256, FAKE, 65535 * 256, 256, B.GQ_BF16, 3, FAKE, FAKE, pages, lay,
                          None) == B.GQ_ERR_INVALID_ARG
    assert L.gq_kv4_read(FAKE, pages, lay, FAKE, 3, FAKE, FAKE, B.GQ_F32, None) == B.GQ_ERR_INVALID_ARG
    a = attn_args(layout=lay, n_pages=pages, q_heads=65535)
    assert L.gq_kv4_attention(ctypes.byref(a), FAKE, 1 << 30, None) == B.GQ_ERR_INVALID_ARG


def test_the_largest_cache_that_fits_is_accepted():
    n = ctypes.c_size_t()
    pages = ((1 << 63) - 1) // PAGE
    assert B.lib().gq_kv4_cache_bytes(pages, layout(**WIDE), ctypes.byref(n)) == B.GQ_OK
    assert n.value == pages * PAGE


def workspace(**kw):
    n = ctypes.c_size_t()
    assert B.lib().gq_kv4_attention_workspace_size(ctypes.byref(attn_args(**kw)), ctypes.byref(n)) == B.GQ_OK
    return n.value


def test_workgroups_do_not_run_out_at_the_largest_sizes():
    # tiles of the split were counted past 63 bits: 8 workgroups for the whole call
    plain = workspace(layout=layout(kv_heads=1), q_heads=1, batch=64, q_tokens=64 * 4096, q_starts=FAKE,
                      max_q_len=4096, max_kv_len=4096)
    for max_kv in (0, 1, 1 << 20, 1 << 30):
        huge = workspace(layout=layout(kv_heads=65535), q_heads=65535, batch=1 << 24, q_tokens=1, q_starts=FAKE,
                         max_q_len=1 << 30, max_kv_len=max_kv)
        assert huge == plain


def test_few_row_tiles_are_split_from_fewer_keys_on():
    # 512 keys and 8 more per row tile, 1024 at most, go to one workgroup without scratch
    for batch, limit in ((1, 576), (4, 768), (8, 1024), (100, 1024)):
        a = dict(batch=batch, q_tokens=batch, max_q_len=1)
        assert workspace(max_kv_len=limit, **a) == 0 and workspace(max_kv_len=limit + 1, **a) > 0
