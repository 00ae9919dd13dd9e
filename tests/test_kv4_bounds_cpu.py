"""The bounds of the prompt tests say something: results that are off by what a
wrong kernel would be off by (planted in the oracle) exceed them, and correctly
rounded results do not."""
import pytest
import torch

from kv4_bounds import exact_key_bounds, uniform_bounds
from kv4_util import attention64, quantise64

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def problem(d, g, dtype, n=120, kv=333, h=1, r=2, seed=3):
    gen = torch.Generator().manual_seed(seed)
    rows = lambda t, heads: (torch.randn(t, heads, d, generator=gen) * torch.exp(torch.randn(t, heads, 1, generator=gen))
                             + 0.5 * torch.randn(heads, d, generator=gen)).to(dtype)
    k, sk, _ = quantise64(rows(kv, h), g, False)
    v, sv, _ = quantise64(rows(kv, h), g, False)
    q = (1.5 * torch.randn(n, h * r, d, generator=gen)).to(dtype).double()
    return q, k, v, sk.amax(-1), sv.amax(-1)


def worst(q, k, v, sk, sv, dtype, window=0, wrong=lambda k, v, o: (k, v, o)):
    """Largest error / bound of the outputs and of lse with a mistake planted."""
    n, kv, scale = q.shape[0], k.shape[0], q.shape[2] ** -0.5
    o, lse, p = attention64(q, k, v, n, kv, True, window, scale)
    tol, lse_tol = exact_key_bounds(q, k, v, sk, sv, o, lse, p, scale, dtype, "many")
    k2, v2, _ = wrong(k, v, None)
    got, gl, _ = attention64(q, k2, v2, n, kv, True, window, scale)
    got = wrong(k2, v2, got)[2].to(dtype).double()
    return float(((got - o).abs() / tol).max()), float(((gl - lse).abs() / lse_tol).max())


def noise(k, v, o):
    gen = torch.Generator().manual_seed(1)
    return k, v, o if o is None else o * (1 + 0.05 * torch.randn(o.shape, generator=gen, dtype=torch.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g", [(64, 64), (128, 32), (256, 128)])
def test_bounds_tell_right_from_wrong(d, g, dtype):
    a = problem(d, g, DT[dtype])
    assert max(worst(*a, DT[dtype])) <= 1.0
    assert worst(*a, DT[dtype], wrong=lambda k, v, o: (k, 1.03 * v, o))[0] > 1.0
    assert worst(*a, DT[dtype], wrong=noise)[0] > 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g", [(64, 64), (128, 32), (256, 128)])
def test_a_window_of_one_key_shows_rounded_keys(d, g, dtype):
    # lse is the score of one key then, and no other key averages its error out
    a = problem(d, g, DT[dtype])
    assert max(worst(*a, DT[dtype], window=1)) <= 1.0
    assert worst(*a, DT[dtype], window=1, wrong=lambda k, v, o: (k.half().double(), v, o))[1] > 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g", [(64, 64), (128, 32), (256, 128)])
def test_equal_scores_show_a_lost_key_and_rounded_values(d, g, dtype):
    # every key has the same weight then, so one that is lost is missed whichever it is
    dt = DT[dtype]
    q, k, v, _, _ = problem(d, g, dt)
    q, n, kv = torch.zeros_like(q), q.shape[0], k.shape[0]
    attend = lambda v, dead=None: attention64(q, k, v, n, kv, True, 0, 1.0, dead)
    o, _, p = attend(v)
    tol = uniform_bounds(v, p, o, dt)
    worst = lambda got: float(((got.to(dt).double() - o).abs() / tol).max())
    assert worst(o) <= 1.0
    for lost in (0, 150, 212):
        assert worst(attend(v, torch.arange(kv) == lost)[0]) > 1.0
    if dt == torch.float16:                     # fp16 results take the values whole
        assert worst(attend(v.half().double())[0]) > 1.0
