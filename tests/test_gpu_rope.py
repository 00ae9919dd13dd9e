"""Rotary positions on the GPU against the definition in 64 bits.

Tolerance: with m the amplitude and |a| + |b| the pair's elements, the sines and
cosines are off by 2^-23 (a turn's fraction, its rest and the function: an ulp of 1
together), products and sums by 3 roundings of 2^-24: 2^-21 m (|a| + |b|) in all, and
half a step of the result's type.  Angles of position p: 2^-52 |p f| more.
"""
import math

import pytest
import torch

from gpu_util import announce, device
from w4a16_dequant_gemm_group_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def turn64(x, pos, f, inter, m, inverse):
    """The rotation in float64, and |a| + |b| of each element's pair (0 behind rot_dim)."""
    x = x.double()
    rot = 2 * f.numel()
    a = pos.double()[:, None, None] * f.double()
    c, s = m * torch.cos(a), m * torch.sin(a) * (-1 if inverse else 1)
    y, size = x.clone(), torch.zeros_like(x)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    size[..., i] = size[..., j] = x[..., i].abs() + x[..., j].abs()
    return y, size


def tolerance(y, size, dtype, m, angle):
    t = (2.0 ** -21 + 2.0 ** -52 * angle) * m * size
    t = t + torch.finfo(dtype).eps / 2 * (y.abs() + t)
    return t + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134)     # below the normal range


def check(x, pos, f, inter=False, m=1.0, inverse=False, **kw):
    y = B.gq_rope(x, pos, f, inter, m, inverse, **kw)
    torch.cuda.synchronize()
    ref, size = turn64(x.cpu(), pos.cpu(), f.cpu(), inter, m, inverse)
    angle = float((pos.abs().double().max() * f.abs().max())) if pos.numel() else 0.0
    err = (y.cpu().double() - ref).abs() - tolerance(ref, size, x.dtype, m, angle)
    assert float(err.max()) <= 0, f"over the tolerance by {float(err.max()):.3e}"
    rot = 2 * f.numel()
    assert torch.equal(y[..., rot:], x[..., rot:])
    return y


def freqs(rot, base=10000.0):
    return B.gq_rope_frequencies(rot, base, device=device())[0]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens,heads,d,rot", [
    (1, 1, 2, 2), (1, 40, 128, 128), (3, 5, 96, 64), (7, 3, 80, 20), (5, 2, 1024, 1024), (257, 6, 64, 64), (2, 300, 64, 32),
    (33, 1, 256, 184), (4099, 4, 32, 16), (9, 7, 10, 6), (1, 65536, 2, 2)])
def test_sizes(dtype, inter, tokens, heads, d, rot):
    announce(f"rope {dtype} interleaved={inter} {tokens}x{heads}x{d} rot {rot}")
    g = torch.Generator().manual_seed(tokens + d)
    x = torch.randn(tokens, heads, d, generator=g).to(DT[dtype]).to(device())
    pos = torch.randint(0, 5000, (tokens,), generator=g).to(device())
    check(x, pos, freqs(rot), inter)
    check(x, pos, freqs(rot), inter, 1.25, True)


@pytest.mark.parametrize("inter", [False, True])
def test_positions_far_and_negative(inter):
    x = torch.randn(8, 3, 128, generator=torch.Generator().manual_seed(1)).to(device())
    pos = torch.tensor([0, -1, 1 << 20, -(1 << 20) - 1, (1 << 31) + 7, 1 << 40, -(1 << 33), 131071], device=device())
    f = freqs(128)
    for i in range(8):      # one by one: the tolerance follows the angle
        check(x[i:i + 1], pos[i:i + 1], f, inter)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_views_and_in_place(dtype, inter):
    g = torch.Generator().manual_seed(2)
    full = torch.randn(37, 14, 64, generator=g).to(DT[dtype]).to(device())
    pos, f = torch.arange(37, device=device()), freqs(64)
    y = check(full[:, 3:9], pos, f, inter)                       # heads of a fused projection
    check(full[::5], pos[::5].contiguous(), f, inter)            # every fifth token
    odd = torch.randn(37 * 14 * 66 + 1, generator=g).to(DT[dtype]).to(device())[1:].view(37, 14, 66)[:, :, 1:65]
    check(odd, pos, f, inter)                                    # rows that are not aligned
    part = check(full[:, 3:9], pos, freqs(32), inter)
    out = torch.full((37, 8, 64), 7.0, dtype=DT[dtype], device=device())
    B.gq_rope(full[:, 3:9], pos, f, inter, out=out[:, 1:7])      # into a view
    assert torch.equal(out[:, 1:7], y) and bool((out[:, 0] == 7).all()) and bool((out[:, 7] == 7).all())
    keep = full.clone()
    B.gq_rope(full[:, 3:9], pos, freqs(32), inter, out=full[:, 3:9])
    assert torch.equal(full[:, 3:9], part)
    assert torch.equal(full[:, :3], keep[:, :3]) and torch.equal(full[:, 9:], keep[:, 9:])


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_is_the_gradient(inter):
    """<w, J dx> = <J^T w, dx> for the differences of the forward pass (it is linear), and the
    inverse of an amplitude of 1 turns back."""
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn(19, 4, 96, generator=g).to(device()) for _ in range(2))
    pos, f, m = torch.arange(1000, 1019, device=device()), freqs(64), 1.3
    grad = B.gq_rope(w, pos, f, inter, m, True)
    h = 0.5
    for t, head, c in ((0, 0, 0), (3, 1, 17), (18, 3, 63), (7, 2, 64), (9, 0, 95)):
        d = torch.zeros_like(x)
        d[t, head, c] = h
        diff = (B.gq_rope(x + d, pos, f, inter, m).double() - B.gq_rope(x - d, pos, f, inter, m).double()) / (2 * h)
        # passed through behind rot_dim; the differences of 4 fp32 results of up to |x| + h each
        assert math.isclose(float((diff * w.double()).sum()), float(grad[t, head, c]), abs_tol=2.0 ** -18 * 12 * 6)
    back = B.gq_rope(B.gq_rope(x, pos, f, inter), pos, f, inter, inverse=True)
    assert float((back - x).abs().max()) <= 2 * 2.0 ** -21 * 2 * 2 * float(x.abs().max())


def test_special_values_empty_stream_graph():
    dev = device()
    f = freqs(64)
    x = torch.randn(6, 2, 64, device=dev).bfloat16()
    pos = torch.arange(6, device=dev)
    assert B.gq_rope(x[:0], pos[:0], f).shape == (0, 2, 64)
    assert B.gq_rope(x[:, :0], pos, f).shape == (6, 0, 64)
    x[2, 1, 5] = float("inf")
    x[3, 0, 9] = float("nan")
    y = B.gq_rope(x, pos, f)
    bad = ~torch.isfinite(y.float())
    assert bad[2, 1, [5, 37]].all() and bad[3, 0, [9, 41]].all() and int(bad.sum()) == 4
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = B.gq_rope(x, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(torch.nan_to_num(z), torch.nan_to_num(y))
    x = torch.randn(6, 2, 64, device=dev).bfloat16()
    B.gq_rope(x, pos, f)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.gq_rope(x, pos, f)
    for i in range(4):
        x.copy_(torch.randn(6, 2, 64, device=dev))
        pos += 100
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, B.gq_rope(x, pos, f))


@pytest.mark.parametrize("tokens,heads,ts,hs", [(9, 5, 64, 9 * 64), (2, 3, 48 * 8, 32 * 8), (4, 4, 55 * 8, 22 * 8)])
def test_layouts_of_out(tokens, heads, ts, hs):
    """Rows of out apart from each other in orders other than tokens of heads."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(tokens, heads, 64, generator=g).bfloat16().to(device())
    pos, f = torch.arange(tokens, device=device()), freqs(64)
    size = (tokens - 1) * ts + (heads - 1) * hs + 64
    memory = torch.full((size + 64,), 7.0, dtype=torch.bfloat16, device=device())
    out = memory.as_strided((tokens, heads, 64), (ts, hs, 1))
    B.gq_rope(x, pos, f, out=out)
    assert torch.equal(out, B.gq_rope(x, pos, f))
    assert int((memory == 7).sum()) >= memory.numel() - x.numel() and bool((memory[size:] == 7).all())
    for strides in ((64, 64), (128, 64)):
        with pytest.raises(B.GqError):
            B.gq_rope(x, pos, f, out=memory.as_strided((tokens, heads, 64), strides + (1,)))
