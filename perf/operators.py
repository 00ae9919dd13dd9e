"""The 4-bit key/value cache and the attention over it: what is measured.

Three operators of the library (C ABI in ``include/gq_kv.h``, called through the
binding): writing keys and values into the cache (quantised on the way), reading
them back, and attention of query rows over the cache, for single new tokens and
for whole prompts.  Each case is one call (a write case also reads back what it
wrote, so that its output is the values the cache now stands for).

The plain forms below use elementary torch operations on a plain cache (packed
nibbles, scales and zero points as separate row-major arrays); ``exact`` works
from the definitions in float64 and shares only the random inputs with them.

Sizes: 32 query and 8 key/value heads of 128 are the Llama-3-8B layer that the
bench and the tests use (qkv projection [6144, 4096]); the others are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _attn(name, hq, hkv, d, g, sym, page, dtype, q_lens, kv_lens, window=0, lse=False):
    c = dict(op="attention", hq=hq, hkv=hkv, d=d, g=g, sym=sym, page=page, dtype=dtype,
             q_lens=" ".join(map(str, q_lens)), kv_lens=" ".join(map(str, kv_lens)),
             window=window, lse=lse)
    if name:
        c["name"] = name
    return c


def _store(op, name, tokens, hkv, d, g, sym, page, dtype, scattered):
    c = dict(op=op, tokens=tokens, hkv=hkv, d=d, g=g, sym=sym, page=page, dtype=dtype,
             scattered=scattered)
    if name:
        c["name"] = name
    return c


def _ragged(n, lo, hi, mul):
    """n lengths spread over [lo, hi] by a fixed rule (odd ones among them)."""
    return [lo + (i * mul) % (hi - lo + 1) for i in range(n)]


def listed():
    return [
        # one sequence's next token enters the cache: latency of the smallest call
        _store("write", "write_1tok", 1, 8, 128, 128, False, 16, "bf16", True),
        # the next tokens of a batch of 61 sequences, each on a page of its own
        _store("write", "write_61tok_sym32", 61, 16, 64, 32, True, 16, "f16", True),
        # a long prompt enters the cache, from a position inside a page
        _store("write", "write_prompt_16k", 16381, 8, 128, 64, False, 64, "bf16", False),
        # a shared prefix of 300 tokens is read back
        _store("read", "read_300_g32", 300, 8, 128, 32, False, 32, "bf16", True),
        # a long sequence is read back whole (handing a cache over in 16 bits)
        _store("read", "read_64k", 65536, 8, 128, 128, False, 64, "f16", False),
        # one token over a short context: latency
        _attn("decode_b1_201", 32, 8, 128, 128, False, 16, "bf16", [1], [201]),
        # one token over a very long context: the length has to be split
        _attn("decode_b1_128k", 32, 8, 128, 64, False, 64, "bf16", [1], [131072], lse=True),
        # a serving batch of 64 sequences of uneven lengths, finest groups
        _attn("decode_b64_ragged_g32", 32, 8, 128, 32, False, 16, "bf16", [1] * 64,
              _ragged(64, 1, 8191, 3541)),
        # four tokens a step to be verified, every head with keys of its own
        _attn("verify4_b16_mha64", 16, 16, 64, 64, True, 32, "f16", [4] * 16,
              _ragged(16, 4, 4000, 1777)),
        # a prompt of 4096 tokens over itself
        _attn("prefill_4096", 32, 8, 128, 128, False, 64, "bf16", [4096], [4096]),
        # chunks of several prompts after cached prefixes, one of them a single token
        _attn("prefill_ragged_g32", 32, 8, 128, 32, False, 16, "f16", [1, 700, 333, 64, 905],
              [2500, 700, 5333, 1087, 3001], lse=True),
        # a chunk late in a long text, attention limited to the last 4096 keys, one key head
        _attn("prefill_window_mqa256", 8, 1, 256, 128, False, 64, "bf16", [1023], [30001],
              window=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 96, 128, 128, 128, 256])
    g = rng.choice([x for x in (32, 64, 96, 128) if d % x == 0])
    sym = rng.random() < 0.35
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 4, 7, 8])
    kind = rng.choice(["write", "read", "decode", "decode", "verify", "prefill"])
    if kind in ("write", "read"):
        top = 16384 * 8 * 128 // (hkv * d) * (1 if kind == "write" else 4)
        return _store(kind, None, _log_int(rng, 1, min(top, 32768)), hkv, d, g, sym, page, dtype,
                      rng.random() < 0.5)
    if kind in ("decode", "verify"):
        n = _log_int(rng, 1, 64)
        # sum of lengths at most 256 K tokens of 8 heads of 128
        top = 262144 * 8 * 128 // (hkv * d) // n
        top = min(top, 131072)
        lens = [_log_int(rng, 1, max(16, top)) for _ in range(n)]
        q = [1] * n
        if kind == "verify":
            q = [min(rng.randint(1, 6), x) for x in lens]
        return _attn(None, hq, hkv, d, g, sym, page, dtype, q, lens, lse=rng.random() < 0.5)
    n = rng.randint(1, 5)
    hq = min(hq, 32) // hkv * hkv
    budget = 4096 * 4096 * 32 * 128 // (hq * d)
    q, lens = [], []
    for _ in range(n):
        x = _log_int(rng, 1, 3000 // n)
        past = rng.choice([0, _log_int(rng, 1, 8000)])
        past = min(past, max(0, budget // n // x - x))
        q.append(x)
        lens.append(x + past)
    return _attn(None, hq, hkv, d, g, sym, page, dtype, q, lens,
                 window=rng.choice([0, 0, _log_int(rng, 1, 4000)]), lse=rng.random() < 0.5)


def _lens(case):
    return [int(x) for x in case["q_lens"].split()], [int(x) for x in case["kv_lens"].split()]


def _pairs(case):
    """(query, key) pairs of all sequences, and the keys that any query reads."""
    pairs = keys = 0
    w = case["window"]
    for n, kv in zip(*_lens(case)):
        first = kv - n
        for p in range(first, kv):
            pairs += min(p + 1, w) if w else p + 1
        keys += kv - max(0, first - w + 1) if w else kv
    return pairs, keys


def work(case):
    h, d = case["hkv"], case["d"]
    row = d // 2 + (2 if case["sym"] else 4) * (d // case["g"])   # bytes of one key or value row
    if case["op"] == "attention":
        pairs, keys = _pairs(case)
        n_q = sum(_lens(case)[0])
        io = n_q * case["hq"] * (2 * d * 2 + (4 if case["lse"] else 0))
        return {"bytes": 2 * keys * h * row + io, "flops": 4 * pairs * case["hq"] * d}
    t = case["tokens"]
    values, stored = 2 * t * h * d * 2, 2 * t * h * row
    n = 2 if case["op"] == "write" else 1                        # 16-bit values in and out
    return {"bytes": n * values + stored + 8 * t, "flops": n * 4 * t * h * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _kv(gen, tokens, h, d, dtype):
    """Keys with a per-channel offset and a few large channels, values of uneven
    size from token to token: what a trained layer's projections look like."""
    dev = gen.device
    off = torch.randn(h, d, generator=gen, device=dev)
    gain = torch.ones(h, d, device=dev)
    gain[:, torch.randperm(d, generator=gen, device=dev)[:4]] = 4.0
    k = (torch.randn(tokens, h, d, generator=gen, device=dev) * gain + off).to(dtype)
    size = torch.exp(0.5 * torch.randn(tokens, h, 1, generator=gen, device=dev))
    v = (0.5 * size * torch.randn(tokens, h, d, generator=gen, device=dev)).to(dtype)
    return k, v


def _inputs(case, seed):
    """Random inputs, and where each token lives in the cache (slot numbers)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype, page = DTYPES[case["dtype"]], case["page"]
    if case["op"] != "attention":
        t = case["tokens"]
        k, v = _kv(gen, t, case["hkv"], case["d"], dtype)
        n_pages = -(-t // page) + 2
        if case["scattered"]:
            slots = torch.randperm(n_pages * page, generator=gen, device="cuda")[:t]
        else:                                                    # consecutive positions from 5 on
            table = torch.randperm(n_pages, generator=gen, device="cuda")
            pos = torch.arange(5, 5 + t, device="cuda")
            slots = table[pos // page] * page + pos % page
        return dict(k=k, v=v, slots=slots, n_pages=n_pages)
    q_lens, kv_lens = _lens(case)
    need = [-(-x // page) for x in kv_lens]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    slots = []
    for b, n in enumerate(kv_lens):
        pos = torch.arange(n, device="cuda")
        slots.append(table[b].long()[pos // page] * page + pos % page)
    k, v = _kv(gen, sum(kv_lens), case["hkv"], case["d"], dtype)
    q = (1.5 * torch.randn(sum(q_lens), case["hq"], case["d"], generator=gen, device="cuda")).to(dtype)
    return dict(q=q, k=k, v=v, slots=torch.cat(slots), table=table, n_pages=n_pages)


def prepare(case, seed):
    i = _inputs(case, seed)
    s = dict(case=case, n_pages=i["n_pages"], slots=i["slots"])
    if own:
        from w4a16_dequant_gemm_group_amd import binding as B
        cache = B.gq_kv4_empty(i["n_pages"], case["hkv"], case["d"], case["page"], case["g"],
                               case["sym"], device="cuda")
    else:
        cache = _plain_empty(i["n_pages"] * case["page"], case)
    s["cache"] = cache
    if case["op"] == "write":
        s.update(k=i["k"], v=i["v"])
        return s
    if own:
        B.gq_kv4_write(i["k"], i["v"], cache, i["slots"], case["g"], case["sym"])
    else:
        _plain_write(i["k"], i["v"], cache, i["slots"], case)
    if case["op"] == "attention":
        q_lens, kv_lens = _lens(case)
        starts = [0]
        for n in q_lens:
            starts.append(starts[-1] + n)
        s.update(q=i["q"], table=i["table"], q_lens=q_lens, kv_lens=kv_lens,
                 q_starts_dev=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                 kv_lens_dev=torch.tensor(kv_lens, dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        from w4a16_dequant_gemm_group_amd import binding as B
        g, sym, cache = c["g"], c["sym"], state["cache"]
        if c["op"] == "attention":
            single = max(state["q_lens"]) == 1
            return B.gq_kv4_attention(
                state["q"], cache, state["table"], state["kv_lens_dev"], g, sym,
                q_starts=None if single else state["q_starts_dev"],
                max_q_len=max(state["q_lens"]), max_kv_len=max(state["kv_lens"]),
                causal=True, window=c["window"], return_lse=c["lse"])
        if c["op"] == "write":
            B.gq_kv4_write(state["k"], state["v"], cache, state["slots"], g, sym)
        return B.gq_kv4_read(cache, state["slots"], c["d"], g, sym, out_dtype=DTYPES[c["dtype"]])
    if c["op"] == "attention":
        return _plain_attention(state)
    if c["op"] == "write":
        _plain_write(state["k"], state["v"], state["cache"], state["slots"], c)
    k, v = _plain_read(state["cache"], state["slots"], c)
    return k.to(DTYPES[c["dtype"]]), v.to(DTYPES[c["dtype"]])


def _plain_empty(n_slots, case):
    h, d = case["hkv"], case["d"]
    ng = d // case["g"]
    out = {}
    for x in "kv":
        out[x] = torch.zeros(n_slots, h, d // 2, dtype=torch.uint8, device="cuda")
        out[x + "s"] = torch.zeros(n_slots, h, ng, dtype=torch.float16, device="cuda")
        if not case["sym"]:
            out[x + "z"] = torch.zeros(n_slots, h, ng, dtype=torch.float16, device="cuda")
    return out


def _plain_quantise(x, case):
    """[T, H, D] -> packed nibbles, scales, zero points.  In 64 bits: codes are
    roundings, and a value next to a border must fall on the right side."""
    t, h, d = x.shape
    g = x.double().view(t, h, d // case["g"], case["g"])
    if case["sym"]:
        r = g.abs().amax(-1) / 7
        lo = None
    else:
        lo = g.amin(-1).clamp(max=0)
        r = (g.amax(-1).clamp(min=0) - lo) / 15
    r = torch.where(r > 0, r, 1.0)
    s = r.clamp(max=65504.0).to(torch.float16)
    s = torch.where(s == 0, 2.0 ** -24, s)
    sd = s.double()
    if case["sym"]:
        z = None
        c = torch.round(g / sd[..., None]).clamp(-8, 7) + 8
    else:
        z = torch.round(-lo / sd).clamp(0, 15)
        c = (torch.round(g / sd[..., None]) + z[..., None]).clamp(0, 15)
        z = z.to(torch.float16)
    c = c.to(torch.uint8).view(t, h, d // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), s.to(torch.float16), z


def _plain_write(k, v, cache, slots, case):
    for name, x in (("k", k), ("v", v)):
        codes, s, z = _plain_quantise(x, case)
        cache[name][slots] = codes
        cache[name + "s"][slots] = s
        if z is not None:
            cache[name + "z"][slots] = z


def _plain_read(cache, slots, case):
    """Values of the given slots in float32 (exact: an 11-bit scale times a 5-bit integer)."""
    out = []
    for name in "kv":
        p = cache[name][slots]
        c = torch.stack((p & 15, p >> 4), -1).float()
        t, h = p.shape[:2]
        c = c.view(t, h, case["d"] // case["g"], case["g"])
        z = 8.0 if case["sym"] else cache[name + "z"][slots].float()[..., None]
        out.append(((c - z) * cache[name + "s"][slots].float()[..., None]).view(t, h, case["d"]))
    return out


def _plain_attention(state):
    c = state["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    page, r = c["page"], hq // hkv
    q = state["q"].float() * (1.0 / math.sqrt(d))
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    at = 0
    for b, (n, kv) in enumerate(zip(state["q_lens"], state["kv_lens"])):
        # a window's earliest key, known to the host
        t0 = max(0, kv - n - c["window"] + 1) if c["window"] else 0
        pos = torch.arange(t0, kv, device="cuda")
        slots = state["table"][b].long()[pos // page] * page + pos % page
        k, v = _plain_read(state["cache"], slots, c)
        k = k.permute(1, 2, 0).contiguous()                                   # [hkv, d, kv]
        v = v.transpose(0, 1).contiguous()                                    # [hkv, kv, d]
        # rows (head in group, token) of each key head
        qb = q[at:at + n].view(n, hkv, r, d).permute(1, 2, 0, 3).reshape(hkv, r * n, d)
        s = torch.matmul(qb, k).view(hkv, r, n, kv - t0)
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        hide = pos > p
        if c["window"]:
            hide = hide | (pos <= p - c["window"])
        s = s.masked_fill(hide, float("-inf"))
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m)
        l = e.sum(-1, keepdim=True)
        o = torch.matmul((e / l).view(hkv, r * n, kv - t0), v)
        out[at:at + n] = o.view(hkv, r, n, d).permute(2, 0, 1, 3).reshape(n, hq, d)
        lse[at:at + n] = (m + torch.log(l)).view(hkv, r, n).permute(2, 0, 1).reshape(n, hq)
        at += n
    out = out.to(state["q"].dtype)
    return (out, lse) if c["lse"] else out


# ---------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------

def _exact_values(x, g, sym):
    """What the 4-bit cache stands for when x was written: the nearest multiple of
    the group's stored scale within the code range."""
    shape = x.shape
    x = x.to(torch.float64).reshape(-1, g)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    if sym:
        step = x.abs().max(1).values / 7.0
    else:
        low = torch.minimum(x.min(1).values, zero)
        step = (torch.maximum(x.max(1).values, zero) - low) / 15.0
    step[step == 0] = 1.0
    step = torch.clamp(step, max=65504.0).to(torch.float16).to(torch.float64)
    step[step == 0] = 2.0 ** -24
    n = torch.round(x / step[:, None])
    if sym:
        n = torch.clamp(n, -8, 7)
    else:
        z = torch.clamp(torch.round(-low / step), 0, 15)[:, None]
        n = torch.minimum(torch.maximum(n, -z), 15 - z)
    return (n * step[:, None]).reshape(shape)


def exact(case, seed):
    i = _inputs(case, seed)
    k = _exact_values(i["k"], case["g"], case["sym"])
    v = _exact_values(i["v"], case["g"], case["sym"])
    if case["op"] != "attention":
        return k, v
    q_lens, kv_lens = _lens(case)
    hq, d, w = case["hq"], case["d"], case["window"]
    rep = hq // case["hkv"]
    out = torch.zeros(sum(q_lens), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(q_lens), hq, dtype=torch.float64, device="cuda")
    qa = ka = 0
    for n, kv in zip(q_lens, kv_lens):
        for a in range(0, n, 1024):                              # query blocks bound the memory
            b = min(n, a + 1024)
            last = kv - n + b                                    # keys 0 .. last - 1 can be seen
            i_pos = torch.arange(kv - n + a, last, device="cuda").unsqueeze(1)
            j_pos = torch.arange(last, device="cuda").unsqueeze(0)
            seen = j_pos <= i_pos
            if w:
                seen &= j_pos > i_pos - w
            for h in range(hq):
                logits = i["q"][qa + a:qa + b, h].double() @ k[ka:ka + last, h // rep].T.contiguous()
                logits = torch.where(seen, logits / d ** 0.5, -math.inf)
                norm = torch.logsumexp(logits, 1)
                out[qa + a:qa + b, h] = torch.exp(logits - norm[:, None]) @ v[ka:ka + last, h // rep]
                lse[qa + a:qa + b, h] = norm
        qa, ka = qa + n, ka + kv
    return (out, lse) if case["lse"] else out
