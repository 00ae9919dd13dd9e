"""How far the attention over the 4-bit cache may be off when every key is taken
exactly: bounds per output element and per log-sum-exp, from the roundings alone."""
import torch


def block_scales(s):
    """s [kv, H], the largest scale of each row -> the largest of each row's 16
    neighbours (one sub-block of the cache), none below fp16's normal range."""
    n = s.shape[0]
    pad = torch.cat((s, s.new_zeros(-n % 16, s.shape[1]))).view(-1, 16, s.shape[1])
    return pad.amax(1).clamp(min=2.0 ** -14).repeat_interleave(16, 0)[:n]


def exact_key_bounds(q, k, v, sk, sv, o, lse, p, scale, dtype, kind):
    """q [n, HQ, D], k / v [kv, H, D] the values the cache stands for, sk / sv [kv, H]
    the largest scale of each row (0: a row of zeros), o / lse / p the definition's
    results; all float64.  Keys begin at a multiple of 16 of their page.

    kind: "many" rows per key/value head, "few" rows, or "once": few rows whose
    fp16 weights are carried with what their rounding left.  Counted:
      scores   exact products of q and k^ summed in fp32: 2 D + 16 roundings of
               2^-24 of sum |q k^|; many rows: keys in two fp16 parts, 2^-22 of it, or
               16 halves of 2^-24 at 2^-10 of the largest scale of 16 neighbours.
               An error d_j of the scores moves o by at most sum p_j d_j (|v_j| + |o|)
      weights  one rounding to fp16, 2^-11 ("once": two parts, 2^-21); below fp16's
               normal range half of 2^-24 of a weight times value scale, of which the
               largest is at least 2^11 (many rows: 2^8), times up to 30 for the
               value: 30 n 2^-36 (2^-33) of the largest
      values   many rows with bf16 results: one rounding to fp16, 2^-11; with fp16
               results two parts, 2^-22; either way 2^-30 of the neighbours' scale
      exp2 and the sums: 2^-18 of sum p |v|
      output   half a step of its type
      lse      the scores' and 2^-18 (log2 of a sum of up to 2^27: one step of 2^-19)
    """
    r = q.shape[1] // k.shape[1]
    rep = lambda t: t.repeat_interleave(r, 1)
    n_keys, d = k.shape[0], q.shape[2]
    half = torch.finfo(dtype).eps / 2
    s_abs = scale * torch.einsum("nhd,khd->nhk", q.abs(), rep(k).abs())
    s_err = s_abs * (2 * d + 16) * 2.0 ** -24
    near = rep(block_scales(sv)).T[None]                        # [1, HQ, kv]
    if kind == "many":
        s_err = s_err + 2.0 ** -22 * s_abs
        s_err = s_err + 2.0 ** -30 * scale * q.abs().sum(-1)[..., None] * rep(block_scales(sk)).T[None]
    lse_err = (p * s_err).sum(-1)
    v_abs = rep(v).abs()
    mean_abs = torch.einsum("nhk,khd->nhd", p, v_abs)
    scores = torch.einsum("nhk,khd->nhd", p * s_err, v_abs) + o.abs() * lse_err[..., None]
    rel = (2.0 ** -21 if kind == "once" else 2.0 ** -11) + 2.0 ** -18
    if kind == "many":
        rel += 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    small = 30 * n_keys * 2.0 ** (-33 if kind == "many" else -36) * (p * near).amax(-1) if n_keys else torch.zeros_like(lse)
    if kind == "many":
        small = small + 2.0 ** -30 * (p * near).sum(-1)
    tol = mean_abs * rel + scores + small[..., None]
    tol = tol + half * (o.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    lse_tol = lse_err + 2.0 ** -18 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)
    return tol, lse_tol


def uniform_bounds(v, p, o, dtype):
    """The same where all scores are zero: the weights are powers of two, so only
    values that are not taken whole show besides the output's half step (with bf16
    results of many rows they are rounded to fp16 once, an eighth of that)."""
    mean_abs = torch.einsum("nhk,khd->nhd", p, v.repeat_interleave(p.shape[1] // v.shape[1], 1).abs())
    tol = mean_abs * (2.0 ** -18 + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21))
    return tol + torch.finfo(dtype).eps / 2 * (o.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
