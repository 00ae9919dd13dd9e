"""Attention over the 8-bit cache where scales lie far apart: the references of the softmax
then move by more powers of two than fp32 has; bounds in kv8_util.attention_bounds."""
import pytest
import torch

from gpu_util import announce
from test_gpu_kv8 import Case

pytestmark = pytest.mark.gpu


# one workgroup per row tile (or few), as the lengths ask for, split as far as it goes
BOUNDS = dict(max_kv_len=1), {}, dict(max_kv_len=1 << 20)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("q_len", [1, 10, 20])
@pytest.mark.parametrize("at", [2.0 ** 90, 2.0 ** 100, 2.0 ** 120, -(2.0 ** 120)])
def test_zeros_before_and_behind_large_values(at, q_len, d):
    """Keys of zeros weigh as much as those of large values, whose scale is up to 2^153 theirs:
    in units, waves, runs and workgroups of their own, where references meet."""
    kv = 1040
    k, q = torch.zeros(kv, 1, d), torch.randn(q_len, 2, d, generator=torch.Generator().manual_seed(1))
    for zeros in (slice(0, 32), slice(0, 64), slice(0, 512), slice(0, 1024), slice(1024, kv), slice(512, kv), slice(256, 640)):
        announce(f"zeros {zeros} beside {at} q_len={q_len} d={d}")
        v = torch.full((kv, 1, d), at)
        v[zeros] = 0
        c = Case(2, 1, d, 16, "bf16", [q_len], [kv], k=k, v=v, q=q)
        for most in BOUNDS:
            c.check(causal=False, **most)
            c.check(**most)


@pytest.mark.parametrize("q_len", [1, 10, 20])
def test_scores_and_scales_apart(q_len):
    """Values that shrink and grow along the keys, beside scores that differ: the sums follow
    every step of the reference."""
    kv, d = 1200, 128
    g = torch.Generator().manual_seed(2)
    k, q = torch.randn(kv, 1, d, generator=g), torch.randn(q_len, 2, d, generator=g)
    base, step = torch.randn(kv, 1, d, generator=g), torch.arange(kv)[:, None, None] // 48
    for e in (5 * step - 30, 95 - 5 * step, 120 * (step % 2) - 20, 110 * (step // 8) - 110):
        v = base * 2.0 ** e.float()
        c = Case(2, 1, d, 16, "bf16", [q_len], [kv], k=k, v=v, q=q)
        for most in BOUNDS:
            c.check(**most)


def test_many_sequences_of_zeros_and_large_values():
    """Runs that take several row tiles of several key tiles each."""
    kv, d, n = 576, 64, 12
    g = torch.Generator().manual_seed(3)
    v = torch.full((kv * n, 1, d), 2.0 ** 110)
    for i in range(n):
        v[kv * i:kv * i + 32 * i] = 0
    q = torch.randn(20 * n, 2, d, generator=g)
    Case(2, 1, d, 16, "bf16", [20] * n, [kv] * n, k=torch.zeros(kv * n, 1, d), v=v, q=q).check()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("q_len", [1, 10, 20])
@pytest.mark.parametrize("low,high", [(-84, 84), (-90, 90), (-118, 116), (112, -30)])
def test_small_queries_and_large_keys(low, high, q_len, d):
    """Scores of ordinary size out of factors at the ends of the range, rows of zeros among them."""
    kv = 200
    g = torch.Generator().manual_seed(4)
    k, v = torch.randn(kv, 1, d, generator=g) * 2.0 ** high, torch.randn(kv, 1, d, generator=g)
    q = torch.randn(q_len, 4, d, generator=g) * 2.0 ** low
    scale = d ** -0.5 * 2.0 ** -(low + high)
    for zero in (False, True):
        if zero:
            q[:, 1] = 0
        c = Case(4, 1, d, 16, "bf16", [q_len], [kv], k=k, v=v, q=q)
        c.check(scale=scale)
        c.check(scale=scale, window=20)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len", [1, 10, 20])
def test_scores_as_large_as_they_may_be(q_len, dtype):
    """Scores up to 2^22, where their steps in fp32 are as large as 1/2: the heaviest key is found,
    and what comes out is a mean of the values."""
    kv, d = 700, 64
    g = torch.Generator().manual_seed(5)
    k, v = torch.randn(kv, 1, d, generator=g), torch.randn(kv, 1, d, generator=g)
    q = torch.randn(q_len, 2, d, generator=g)
    most = float((q[:, :, None] * k[None, :, 0][:, None]).sum(-1).abs().max())
    for sign in (1, -1):
        for drift in (0.0, 1.0):
            # with drift: every key a little heavier than the one before
            kk = k * (1 - drift) + drift * (1 + torch.arange(kv)[:, None, None] * 2.0 ** -9).expand(kv, 1, d) / 2.5
            qq = q * (1 - drift) + drift
            top = most if drift == 0 else float((qq[0, 0] * kk[:, 0]).sum(-1).abs().max())
            scale = 0.98 * 2.0 ** 22 / top
            c = Case(2, 1, d, 16, dtype, [q_len], [kv], k=kk, v=v, q=sign * qq)
            for bound in BOUNDS:
                out = c.check(scale=scale, **bound)
                assert bool((out.abs() <= c.v.double().abs().max() * (1 + 2.0 ** -6)).all())
