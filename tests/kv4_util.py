"""Definitions of the 4-bit key/value cache and its attention in 64 bits, for
the tests (CPU tensors, float64 throughout; no code of the library)."""
import math

import torch


def quantise64(x: torch.Tensor, group: int, sym: bool):
    """x [..., D] -> (values, scales [..., D/g], zeros) in float64."""
    shape = x.shape
    g = x.double().reshape(*shape[:-1], shape[-1] // group, group)
    if sym:
        rng, n = g.abs().amax(-1), 7.0
        lo = None
    else:
        lo = g.amin(-1).clamp(max=0.0)
        rng, n = g.amax(-1).clamp(min=0.0) - lo, 15.0
    step = torch.where(rng > 0, rng / n, torch.ones_like(rng))
    # one rounding to fp16, saturated to [2^-24, 65504] (numpy rounds float64 once)
    s = torch.from_numpy(step.clamp(max=65504.0).numpy().astype("float16")).double()
    s = torch.where(s == 0, torch.full_like(s, 2.0 ** -24), s)
    if sym:
        z = torch.full_like(s, 8.0)
    else:
        z = torch.round(-lo / s).clamp(0, 15)
    c = (torch.round(g / s[..., None]) + z[..., None]).clamp(0, 15)
    return ((c - z[..., None]) * s[..., None]).reshape(shape), s, z


def attention64(q, k, v, q_len, kv_len, causal, window, scale, dead=None):
    """One sequence: q [n, HQ, D], k / v [kv, H, D] float64 -> (o, lse, p, s_abs).
    dead [kv] bool: keys that nobody sees.  A row without keys: zeros, -inf."""
    n, hq, d = q.shape
    h = k.shape[1]
    r = hq // h
    kk = k.repeat_interleave(r, 1)
    vv = v.repeat_interleave(r, 1)
    s = scale * torch.einsum("nhd,khd->nhk", q, kk)
    pos = torch.arange(kv_len - q_len, kv_len)[:, None]
    j = torch.arange(kv_len)[None, :]
    seen = torch.ones(n, kv_len, dtype=torch.bool)
    if causal:
        seen &= j <= pos
    if window:
        seen &= j > pos - window
    if dead is not None:
        seen &= ~dead[None, :]
    s = s.masked_fill(~seen[:, None, :], -math.inf)
    lse = torch.logsumexp(s, -1) if kv_len else torch.full((n, hq), -math.inf, dtype=torch.float64)
    p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    o = torch.einsum("nhk,khd->nhd", p, vv)
    return o, lse, p


def attention_bounds(q, k, v, sk, sv, o, lse, p, scale, dtype, fp16_operands):
    """How far the kernels may be off, per output element and per lse.

    q [n, HQ, D], k / v [kv, H, D], sk / sv [kv, H] the largest scale of each
    key's and value's row, all float64.  Counted:
      scores   fp32 sums of D products of q with codes c and zero points z, both
               up to 15 scales: D + 16 roundings of 2^-24 of sum |q| 30 S;
               with fp16 operands also one rounding (2^-11) of each key element
      weights  one rounding of p S to fp16 (2^-11, or 2^-25 of the largest weight
               of the row below fp16's normal range, times 15 codes), doubled
               for the reference being up to 1.1 powers of two off;
               with fp16 operands also one rounding of each value element
      exp2 and the sums of weights: 2^-20 of the result
      output   half a step of its type
    """
    r = q.shape[1] // k.shape[1]
    rep = lambda t: t.repeat_interleave(r, 1)
    d = q.shape[2]
    n_keys = k.shape[0]
    half = torch.finfo(dtype).eps / 2
    qabs = q.abs().sum(-1)                                     # [n, HQ]
    s_err = scale * (d + 16) * 2.0 ** -24 * 30 * qabs[..., None] * rep(sk).T[None]     # [n, HQ, kv]
    if fp16_operands:
        s_err = s_err + 2.0 ** -11 * scale * torch.einsum("nhd,khd->nhk", q.abs(), rep(k).abs())
    s_max = (s_err * (p > 0)).amax(-1) if n_keys else torch.zeros_like(lse)
    mean_abs = torch.einsum("nhk,khd->nhd", p, rep(v).abs())
    top = (p * rep(sv).T[None]).amax(-1) if n_keys else torch.zeros_like(lse)
    rel = (2 if fp16_operands else 1) * 2.0 ** -11 + 2.0 ** -20 + 2 * s_max
    tol = mean_abs * rel[..., None] + (2 * 15 * n_keys * 2.0 ** -25 * top)[..., None]
    tol = tol + half * (o.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    lse_tol = s_max + 2.0 ** -20 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)
    return tol, lse_tol
