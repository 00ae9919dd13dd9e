"""Rotary positions without a GPU: exports, the frequencies against their formulas,
and refusals before any device call."""
import ctypes
import math
import os

import pytest
import torch

from conftest import ROOT
from test_abi import header_functions
from w4a16_dequant_gemm_group_amd import binding as B

FAKE = 4096


def test_exports_every_declared_symbol():
    names = header_functions(os.path.join(ROOT, "include", "gq_rope.h"))
    assert set(names) == set(B.ROPE_EXPORTS) and len(names) == 2
    for n in names:
        assert hasattr(B.lib(), n), n


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (1024, 2.0)])
def test_plain_and_linear(rot, base):
    f, m = B.gq_rope_frequencies(rot, base, device="cpu")
    ref = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    assert m == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, ref, rtol=1e-15, atol=0)
    g, m = B.gq_rope_frequencies(rot, base, "linear", factor=4.0, device="cpu")
    assert m == 1.0 and torch.allclose(g, ref / 4, rtol=1e-15, atol=0)


def test_wavelength():
    f, _ = B.gq_rope_frequencies(128, 500000.0, device="cpu")
    g, m = B.gq_rope_frequencies(128, 500000.0, "wavelength", factor=8.0, original_length=8192, low=1.0, high=4.0,
                                 device="cpu")
    assert m == 1.0
    kinds = set()
    for a, b in zip(f.tolist(), g.tolist()):
        length = 2 * math.pi / a
        if length > 8192:
            want, kind = a / 8, "long"
        elif length < 2048:
            want, kind = a, "short"
        else:
            t = (8192 / length - 1) / 3
            want, kind = (1 - t) * a / 8 + t * a, "between"
        kinds.add(kind)
        assert math.isclose(b, want, rel_tol=1e-14)
    assert kinds == {"long", "short", "between"}


@pytest.mark.parametrize("rot,length", [(64, 4096), (128, 4096), (16, 20)])
def test_yarn(rot, length):
    base, s, slow, fast = 10000.0, 16.0, 1.0, 32.0
    f, _ = B.gq_rope_frequencies(rot, base, device="cpu")
    g, m = B.gq_rope_frequencies(rot, base, "yarn", factor=s, original_length=length, low=slow, high=fast, device="cpu")
    assert math.isclose(m, 0.1 * math.log(s) + 1, rel_tol=1e-15)
    at = lambda n: rot * math.log(length / (2 * math.pi * n)) / (2 * math.log(base))
    lo = min(max(math.floor(at(fast)), 0), rot - 1)
    hi = max(min(math.ceil(at(slow)), rot - 1), lo + 0.001)
    for i, (a, b) in enumerate(zip(f.tolist(), g.tolist())):
        t = 1 - min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert math.isclose(b, (1 - t) * a / s + t * a, rel_tol=1e-14)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=1026), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")),
    dict(scaling="linear", factor=float("inf")), dict(scaling="yarn", factor=2.0, original_length=0.0),
    dict(scaling="wavelength", factor=2.0, original_length=100.0, low=4.0, high=4.0),
    dict(scaling="wavelength", factor=2.0, original_length=100.0, low=0.0, high=4.0),
    dict(scaling="yarn", factor=2.0, original_length=float("inf")), dict(scaling="other"),
])
def test_frequency_refusals(kw):
    with pytest.raises((ValueError, B.GqError)):
        B.gq_rope_frequencies(**{**dict(rot_dim=64, device="cpu"), **kw})


def test_frequency_null():
    s, m = B.GqRopeScaling(0, 1.0, 1.0, 1.0, 2.0), ctypes.c_double()
    f = (ctypes.c_double * 4)()
    L = B.lib()
    assert L.gq_rope_frequencies(8, 10000.0, s, None, ctypes.byref(m)) == B.GQ_ERR_INVALID_ARG
    assert L.gq_rope_frequencies(8, 10000.0, s, f, None) == B.GQ_ERR_INVALID_ARG
    s.kind = 9
    assert L.gq_rope_frequencies(8, 10000.0, s, f, ctypes.byref(m)) == B.GQ_ERR_INVALID_ARG


def args(**kw):
    a = dict(x=FAKE, x_token_stride=1024, x_head_stride=128, out=2 * FAKE, out_token_stride=1024, out_head_stride=128,
             dtype=B.GQ_BF16, tokens=3, heads=8, head_dim=128, rot_dim=128, positions=FAKE, freqs=FAKE, amplitude=1.0,
             interleaved=0, inverse=0)
    a.update(kw)
    return ctypes.byref(B.GqRopeArgs(*(a[f] for f, _ in B.GqRopeArgs._fields_)))


def test_refusals():
    L = B.lib()
    for kw in (dict(x=None), dict(out=None), dict(positions=None), dict(freqs=None), dict(dtype=9), dict(tokens=-1),
               dict(tokens=(1 << 30) + 1), dict(heads=-1), dict(heads=65537), dict(head_dim=127), dict(head_dim=0),
               dict(head_dim=1026), dict(rot_dim=0), dict(rot_dim=130), dict(rot_dim=63),
               dict(x_token_stride=(1 << 40) + 1), dict(out_head_stride=-(1 << 40) - 1),
               dict(amplitude=float("nan")), dict(amplitude=float("inf")), dict(interleaved=2), dict(inverse=-1),
               dict(out=FAKE, out_token_stride=2048), dict(out=FAKE, out_head_stride=256),
               # rows that overlap
               dict(out_token_stride=0), dict(out_head_stride=0), dict(out_head_stride=-127),
               dict(out=FAKE, x_token_stride=0, out_token_stride=0)):
        assert L.gq_rope(args(**kw), None) == B.GQ_ERR_INVALID_ARG, kw
    for kw in (dict(x=FAKE + 1), dict(out=FAKE + 1), dict(positions=FAKE + 4), dict(freqs=FAKE + 4),
               dict(dtype=B.GQ_F32, x=FAKE + 2)):
        assert L.gq_rope(args(**kw), None) == B.GQ_ERR_MISALIGNED, kw
    assert L.gq_rope(None, None) == B.GQ_ERR_INVALID_ARG
    assert L.gq_rope(args(tokens=0, x=None, out=None), None) == B.GQ_OK
    assert L.gq_rope(args(heads=0, x=None, out=None), None) == B.GQ_OK


@pytest.mark.parametrize("tokens,heads,d,ts,hs", [
    (2, 2, 128, 128, 128), (3, 8, 128, 128, 128), (3, 8, 128, 256, 128), (3, 8, 128, 1023, 128), (8, 3, 128, 128, 1023),
    (3, 8, 128, 896, 128), (2, 9, 64, 512, 64), (2, 2, 128, 128, -128), (3, 8, 128, -1000, 128), (9, 3, 2, 2, 16),
    (4, 4, 10, 35, 24), (1 << 30, 65536, 2, (1 << 17) - 1, 2), (1 << 30, 65536, 2, 1 << 40, (1 << 40) - 1),
    (1 << 30, 65536, 2, 4, 65536 * 4 + 1)])
def test_rows_of_out_that_overlap(tokens, heads, d, ts, hs):
    a = dict(tokens=tokens, heads=heads, head_dim=d, rot_dim=d, out_token_stride=ts, out_head_stride=hs)
    assert B.lib().gq_rope(args(**a, positions=FAKE + 4), None) == B.GQ_ERR_INVALID_ARG


@pytest.mark.parametrize("tokens,heads,d,ts,hs", [
    (3, 8, 128, 1024, 128), (3, 8, 128, 128, 384), (3, 8, 128, -1024, -128), (1, 8, 128, 0, 128), (3, 1, 128, 128, 0),
    (2, 2, 128, 384, 256), (2, 2, 128, 256, 384), (4, 4, 10, 55, 22), (2, 3, 10, 36, 24), (1 << 30, 65536, 2, 1 << 17, 2),
    (1 << 30, 256, 2, 2, 1 << 31), (1 << 30, 65536, 2, 1 << 40, 2)])
def test_rows_of_out_apart(tokens, heads, d, ts, hs):
    """Rows that do not overlap, in whatever order they lie, pass the check: the call is refused
    for what is checked behind it, before anything is launched."""
    a = dict(tokens=tokens, heads=heads, head_dim=d, rot_dim=d, out_token_stride=ts, out_head_stride=hs)
    assert B.lib().gq_rope(args(**a, positions=FAKE + 4), None) == B.GQ_ERR_MISALIGNED


def test_binding_checks():
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    pos, f = torch.zeros(3, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    for a, exc in [((x.double(), pos, f), TypeError), ((x[0], pos, f), ValueError),
                   ((x, pos[:2], f), ValueError), ((x, pos.int(), f), TypeError), ((x, pos, f.float()), TypeError),
                   ((x, pos, f[:0]), ValueError), ((x, pos, torch.zeros(33, dtype=torch.float64)), ValueError),
                   ((x.transpose(1, 2), pos, f), ValueError), (([1], pos, f), TypeError),
                   ((x, pos, f), ValueError)]:       # the last: not on a GPU
        with pytest.raises(exc):
            B.gq_rope(*a)
    with pytest.raises(ValueError):
        B.gq_rope(x, pos, f, out=torch.zeros(3, 4, 32, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        B.gq_rope(x, pos, f, out=x.float())
