"""Definitions of the 8-bit key/value cache, its attention and the choice of pages in
64 bits, for the tests (CPU tensors, float64 throughout; no code of the library)."""
import math

import torch

LEAST = 2.0 ** -40


def scale_of(x):
    """Scale that the values x of one block ask for: one rounding to fp32."""
    m = x.abs().max().double() / 127 if x.numel() else torch.zeros((), dtype=torch.float64)
    return max(float(m.to(torch.float32)), LEAST)


class Blocks:
    """One sequence's keys (or values) of one head as the cache holds them: codes and
    scales of blocks of 16, after any number of calls of `append`."""

    def __init__(self, d):
        self.codes = torch.zeros(0, d, dtype=torch.float64)
        self.scales = []

    def append(self, x, start=None):
        """x [n, d] at positions start .. (default: behind what is there)."""
        x = torch.nan_to_num(x.double(), nan=0.0, posinf=float(torch.finfo(x.dtype).max),
                             neginf=float(torch.finfo(x.dtype).min))
        start = self.codes.shape[0] if start is None else start
        self.codes = self.codes[:start].clone()
        del self.scales[-(-start // 16):]
        at = 0
        while at < x.shape[0]:
            pos = start + at
            n = min(16 - pos % 16, x.shape[0] - at)
            part = x[at:at + n]
            s = scale_of(part)
            if pos % 16:
                old = self.scales[-1]
                s = max(s, old)
                b = pos // 16 * 16
                self.codes[b:] = torch.round(self.codes[b:] * old / s)
                self.scales[-1] = s
            else:
                self.scales.append(s)
            self.codes = torch.cat((self.codes, torch.round(part / s).clamp(-127, 127)))
            at += n
        return self

    def scale_rows(self):
        return torch.tensor(self.scales, dtype=torch.float64).repeat_interleave(16)[:self.codes.shape[0]]

    def values(self):
        return self.codes * self.scale_rows()[:, None]


def cached(x, cuts=None):
    """x [n, heads, d] appended in calls that end at `cuts`: (values, scales [n, heads])."""
    ends = list(cuts or []) + [x.shape[0]]
    vals, scales = [], []
    for h in range(x.shape[1]):
        b, at = Blocks(x.shape[2]), 0
        for e in ends:
            b.append(x[at:e, h])
            at = e
        vals.append(b.values())
        scales.append(b.scale_rows())
    return torch.stack(vals, 1), torch.stack(scales, 1)


def attention_bounds(q, k, v, sk, sv, o, lse, p, scale, dtype, rest):
    """How far the kernels may be off, per output element and per lse.

    q [n, HQ, D], k / v [kv, H, D], sk / sv [kv, H] scales, o, lse, p of the definition,
    all float64.  Counted, with room for the result's own rounding at the end:
      scores   fp32 sums of D exact products of q and codes (127 scales at most), their
               factor and the exponent's argument: D + 16 roundings of 2^-24 of
               127 S sum |q|; log2 of the value scale enters the exponent of weight and sum
               alike, 2^-24 of up to 2^7 and of the score itself
      weights  p S_V rounded to fp16: 2^-11 (rest: what it leaves is carried too, 2^-22),
               or half a subnormal step, 2^-25, where the row's largest is at least 2^8: of
               it, times 127 codes, for every key
      exp2 and the sums of weights: 2^-20 of the result
      output   half a step of its type
    """
    r = q.shape[1] // k.shape[1]
    rep = lambda t: t.repeat_interleave(r, 1)
    d, n_keys = q.shape[2], k.shape[0]
    half = torch.finfo(dtype).eps / 2
    qabs = q.abs().sum(-1)
    s_err = scale * (d + 16) * 2.0 ** -24 * 127 * qabs[..., None] * rep(sk).T[None]
    lv = 2.0 ** -24 * 128
    s_max = (s_err * (p > 0)).amax(-1) if n_keys else torch.zeros_like(lse)
    mean_abs = torch.matmul(p.permute(1, 0, 2), rep(v).abs().permute(1, 0, 2).contiguous()).permute(1, 0, 2)
    top = (p * rep(sv).T[None]).amax(-1) if n_keys else torch.zeros_like(lse)
    rel = (2.0 ** -22 if rest else 2.0 ** -11) + 2.0 ** -20 + 2 * s_max + lv
    tol = mean_abs * rel[..., None] + (127 * n_keys * 2.0 ** -33 * top)[..., None]
    tol = tol + half * (o.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    lse_tol = s_max + lv + 2.0 ** -20 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)
    return tol, lse_tol


def select64(q, lo, hi, p, page, keep, first, last, dead=()):
    """One query q [HQ, D] at position p over bounds lo / hi [pages, H, D], float64: per
    key/value head the chosen page places, ascending, and the keys they hold."""
    n, h = p // page + 1, lo.shape[1]
    r = q.shape[0] // h
    out = []
    for x in range(h):
        score = []
        for j in range(n):
            best = -math.inf
            for y in range(x * r, (x + 1) * r):
                s = float(torch.maximum(q[y] * lo[j, x], q[y] * hi[j, x]).sum())
                if s > best:
                    best = s
            score.append(-math.inf if j in dead else best)
        must = [j for j in range(n) if j < first or j >= n - last]
        rest = sorted(set(range(n)) - set(must), key=lambda j: (-score[j], j))
        out.append(sorted((must + rest)[:min(keep, n)]) if n > keep else list(range(n)))
    return out, (min(n, keep) - 1) * page + p % page + 1
