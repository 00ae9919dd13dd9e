"""Attention over the 4-bit cache within bounds that take every key exactly: all
rows, rows that see one key, rows whose keys all weigh the same."""
import math

import pytest
import torch

from gpu_util import announce
from kv4_bounds import exact_key_bounds, uniform_bounds
from kv4_util import attention64
from test_gpu_kv4 import LAYOUTS, Problem, announce_case

pytestmark = pytest.mark.gpu


def check_exact_keys(p, out, lse, window=0, scale=None, what=""):
    scale = p.d ** -0.5 if scale is None else scale
    many = max(p.q_lens) * p.r > 32
    qa = ka = 0
    worst = worst_l = 0.0
    for n, kv in zip(p.q_lens, p.kv_lens):
        q, k, v = p.q[qa:qa + n].double(), p.k[ka:ka + kv], p.v[ka:ka + kv]
        o, l, w = attention64(q, k, v, n, kv, True, window, scale)
        once = p.dt == torch.float16 and max(p.q_lens) * p.r <= 16 and n * p.r <= 8
        tol, ltol = exact_key_bounds(q, k, v, p.sk[ka:ka + kv], p.sv[ka:ka + kv], o, l, w, scale, p.dt,
                                     "many" if many else "once" if once else "few")
        got, gl = out[qa:qa + n].cpu().double(), lse[qa:qa + n].cpu().double()
        empty = l == -math.inf
        assert torch.equal(gl == -math.inf, empty) and not got[empty].any()
        if (~empty).any():
            worst = max(worst, float(((got - o).abs() / tol)[~empty].max()))
            worst_l = max(worst_l, float(((gl - l).abs() / ltol)[~empty].max()))
        assert torch.isfinite(got).all()
        qa, ka = qa + n, ka + kv
    announce(f"{what}: error / bound {worst:.3f}, lse {worst_l:.3f}")
    assert worst <= 1.0 and worst_l <= 1.0


def check_equal_weights(p, out, what):
    qa = ka = 0
    worst = 0.0
    for n, kv in zip(p.q_lens, p.kv_lens):
        v = p.v[ka:ka + kv]
        o, l, w = attention64(torch.zeros(n, p.h * p.r, p.d, dtype=torch.float64), p.k[ka:ka + kv], v, n, kv, True, 0, 1.0)
        err = (out[qa:qa + n].cpu().double() - o).abs()
        if n and kv:
            worst = max(worst, float((err / uniform_bounds(v, w, o, p.dt)).nan_to_num(nan=0.0).max()))
        qa, ka = qa + n, ka + kv
    announce(f"{what}: error / bound {worst:.3f}")
    assert worst <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g,sym", LAYOUTS)
def test_prompts_take_keys_exactly(d, g, sym, dtype):
    p = Problem(d * 7 + g, d, g, sym, 16, dtype, 2, 2, [150, 1, 0, 65, 200], [150, 40, 9, 1100, 333])
    announce_case(p, "prompts")
    check_exact_keys(p, *p.run(), what="prompts")
    check_exact_keys(p, *p.run(window=1), window=1, what="prompts, one key each")
    check_equal_weights(p, p.run(q=torch.zeros_like(p.q).cuda())[0], "prompts, equal weights")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g,sym", LAYOUTS)
def test_few_rows_take_keys_exactly(d, g, sym, dtype):
    for q_lens, r in (([1] * 6, 4), ([6, 1, 5, 0, 2, 3], 4)):
        p = Problem(d * 11 + g + r, d, g, sym, 16, dtype, 2, r, q_lens, [1, 40, 333, 9, 1500, 128])
        announce_case(p, "few rows")
        check_exact_keys(p, *p.run(), what="few rows")
        check_exact_keys(p, *p.run(window=1) if max(q_lens) > 1 else p.run(starts=p.starts, window=1), window=1,
                         what="few rows, one key each")
