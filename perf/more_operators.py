"""Rotary positions, an 8-bit key/value cache with its attention, and attention
over pages that a cheap score selects: what is measured.

The operators of one decode step or prompt around the cache (C ABI in
``include/gq_rope.h`` and ``include/gq_kv8.h``, called through the binding):
rotating queries and keys by their positions, appending keys and values to a cache
held in 8 bits with one scale for each block of 16 tokens and head, attention over
that cache, and the choice of a few pages per query and key/value head by bounds
that the cache keeps of each page's keys, with the attention over those pages.

The plain forms below use elementary torch operations on a plain cache (codes and
scales as separate row-major arrays); ``exact`` works from the definitions in
float64 and shares only the random inputs with them.

Sizes: 32 query and 8 key/value heads of 128 are the Llama-3-8B layer that the
bench and the tests use (qkv projection [6144, 4096]); the others are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 16                 # tokens that share a scale
LEAST = 2.0 ** -40         # least scale of a block


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _named(name, **c):
    if name:
        c["name"] = name
    return c


def _text(lens):
    return " ".join(map(str, lens))


def _rope(name, tokens, heads, rest, d, rot, dtype, interleaved, inverse, scaling, top):
    """`heads` of the heads + rest heads of a fused projection are rotated; positions up to `top`."""
    return _named(name, op="rope", tokens=tokens, heads=heads, rest=rest, d=d, rot=rot, dtype=dtype,
                  interleaved=interleaved, inverse=inverse, scaling=scaling, top=top)


def _append(name, hkv, d, page, dtype, new, old):
    return _named(name, op="append", hkv=hkv, d=d, page=page, dtype=dtype, new=_text(new), old=_text(old))


def _attn(name, hq, hkv, d, page, dtype, q_lens, kv_lens, window=0, lse=False):
    return _named(name, op="attention", hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, q_lens=_text(q_lens),
                  kv_lens=_text(kv_lens), window=window, lse=lse)


def _sparse(name, hq, hkv, d, page, dtype, q_lens, kv_lens, keep, first, last):
    """`keep` pages a query (at least first + last), its first `first` and last `last` always among them."""
    return _named(name, op="sparse", hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, q_lens=_text(q_lens),
                  kv_lens=_text(kv_lens), keep=keep, first=first, last=last)


def _ragged(n, lo, hi, mul):
    """n lengths spread over [lo, hi] by a fixed rule (odd ones among them)."""
    return [lo + (i * mul) % (hi - lo + 1) for i in range(n)]


def listed():
    return [
        # the next token's queries and keys, a slice of the fused projection's output: latency
        _rope("rope_1tok", 1, 40, 8, 128, 128, "bf16", False, False, "wavelength", 8191),
        # the same for a long prompt
        _rope("rope_prompt_8k", 8191, 40, 8, 128, 128, "bf16", False, False, "none", 8190),
        # gradients of a training batch whose heads are rotated in part, in pairs of neighbours
        _rope("rope_grad_part", 4099, 20, 0, 96, 64, "f16", True, True, "yarn", 131071),
        # one sequence's next token enters the cache: latency
        _append("append_1tok", 8, 128, 16, "bf16", [1], [200]),
        # several prompts enter the cache in one call, some behind what is there already
        _append("append_prompts_16k", 8, 128, 64, "bf16", [9001, 5, 6200, 1, 1177], [0, 1000, 37, 16, 2051]),
        # one token over a short context: latency
        _attn("attn_b1_201", 32, 8, 128, 16, "bf16", [1], [201]),
        # one token over a very long context
        _attn("attn_b1_128k", 32, 8, 128, 64, "bf16", [1], [131071], lse=True),
        # a serving batch of 64 sequences of uneven lengths
        _attn("attn_b64_ragged", 32, 8, 128, 16, "bf16", [1] * 64, _ragged(64, 1, 8191, 3541)),
        # a prompt of 4096 tokens over itself
        _attn("attn_prompt_4096", 32, 8, 128, 64, "bf16", [4096], [4096]),
        # chunks of several prompts behind cached prefixes, heads of 96, a window of 2000 keys
        _attn("attn_chunks_f16_96", 24, 6, 96, 32, "f16", [1, 700, 333, 64, 905], [2500, 700, 5333, 1087, 3001],
              window=2000, lse=True),
        # one token over a very long context, of which 32 pages of 64 are read
        _sparse("sparse_b1_128k", 32, 8, 128, 64, "bf16", [1], [131071], 32, 1, 2),
        # drafted tokens of 16 long sequences, each token with pages of its own
        _sparse("sparse_b16_draft", 16, 4, 64, 16, "f16", [1, 2, 3, 4] * 4, _ragged(16, 40, 16000, 7907), 48, 2, 4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 96, 128, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 4, 7, 8])
    kind = rng.choice(["rope", "append", "decode", "verify", "prompt", "sparse", "sparse"])
    if kind == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2, rng.randrange(2, d + 1, 2)])
        heads, rest = rng.randint(1, 48), rng.choice([0, 0, 8, 16])
        tokens = _log_int(rng, 1, min(32768, 8191 * 40 * 128 // (heads * d)))
        dtype = rng.choice(["bf16", "f16", "f32"])
        return _rope(None, tokens, heads, rest, d, rot, dtype, rng.random() < 0.5, rng.random() < 0.4,
                     rng.choice(["none", "linear", "wavelength", "yarn"]), _log_int(rng, 100, 1 << 20))
    if kind == "append":
        n = _log_int(rng, 1, 64)
        top = 16384 * 8 * 128 // (hkv * d) // n
        new = [_log_int(rng, 1, max(2, top)) for _ in range(n)] if rng.random() < 0.7 else [1] * n
        return _append(None, hkv, d, page, dtype, new, [rng.choice([0, rng.randint(1, 3000)]) for _ in range(n)])
    if kind in ("decode", "verify"):
        n = _log_int(rng, 1, 64)
        top = min(262144 * 8 * 128 // (hkv * d) // n, 131072)
        lens = [_log_int(rng, 1, max(16, top)) for _ in range(n)]
        q = [1] * n if kind == "decode" else [min(rng.randint(1, 6), x) for x in lens]
        return _attn(None, hq, hkv, d, page, dtype, q, lens, lse=rng.random() < 0.5)
    if kind == "sparse":
        n = _log_int(rng, 1, 32)
        top = min(262144 * 8 * 128 // (hkv * d) // n, 131072)
        lens = [_log_int(rng, 1, max(16, top)) for _ in range(n)]
        q = [1] * n if rng.random() < 0.6 else [min(rng.randint(1, 4), x) for x in lens]
        keep = _log_int(rng, 4, max(5, min(96, 4096 // page)))
        first, last = rng.randint(0, 2), rng.randint(1, 2)
        return _sparse(None, hq, hkv, d, page, dtype, q, lens, keep, first, last)
    hq = min(hq, 32) // hkv * hkv
    n = rng.randint(1, 5)
    budget = 4096 * 4096 * 32 * 128 // (hq * d)
    q, lens = [], []
    for _ in range(n):
        x = _log_int(rng, 1, 3000 // n)
        past = rng.choice([0, _log_int(rng, 1, 8000)])
        past = min(past, max(0, budget // n // x - x))
        q.append(x)
        lens.append(x + past)
    return _attn(None, hq, hkv, d, page, dtype, q, lens, window=rng.choice([0, 0, _log_int(rng, 1, 4000)]),
                 lse=rng.random() < 0.5)


def _ints(case, key):
    return [int(x) for x in case[key].split()]


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * case["d"] * size + 8 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    h, d, page = case["hkv"], case["d"], case["page"]
    row = 2 * (d + 4 / BLOCK)                                   # bytes of one key and value in the cache
    if op == "append":
        new, old = _ints(case, "new"), _ints(case, "old")
        n = sum(new)
        back = sum(m + o % BLOCK for m, o in zip(new, old))     # read back: the blocks that the call touched
        pages = sum((o + m - 1) // page - o // page + 1 for m, o in zip(new, old))
        return {"bytes": int(n * h * (4 * d + row) + back * h * (4 * d + row) + 8 * back + pages * h * 4 * d),
                "flops": (n + back) * h * 4 * d}
    q_lens, kv_lens = _ints(case, "q_lens"), _ints(case, "kv_lens")
    io = sum(q_lens) * case["hq"] * 2 * d * 2
    if op == "attention":
        pairs = keys = 0
        w = case["window"]
        for n, kv in zip(q_lens, kv_lens):
            for p in range(kv - n, kv):
                pairs += min(p + 1, w) if w else p + 1
            keys += kv - max(0, kv - n - w + 1) if w else kv
        return {"bytes": int(keys * h * row + io + (4 * sum(q_lens) * case["hq"] if case["lse"] else 0)),
                "flops": 4 * pairs * case["hq"] * d}
    # sparse: all bounds of a sequence once, and the keys of as many pages as one query takes
    bounds = keys = flops = 0
    for n, kv in zip(q_lens, kv_lens):
        bounds += -(-kv // page) * h * 4 * d
        keys += _seen(kv - 1, case)
        for p in range(kv - n, kv):
            flops += (p // page + 1) * case["hq"] * 4 * d + 4 * _seen(p, case) * case["hq"] * d
    return {"bytes": int(bounds + keys * h * row + io + 4 * sum(q_lens) * (h * case["keep"] + 1)), "flops": flops}


def _seen(p, case):
    """Keys that a query at position p reads of the pages it keeps."""
    page = case["page"]
    return (min(p // page + 1, case["keep"]) - 1) * page + p % page + 1


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


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


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _page_table(gen, lens, page):
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, n_pages


def _inputs(case, seed):
    gen = _generator(seed)
    dtype, d = DTYPES[case["dtype"]], case["d"]
    if case["op"] == "rope":
        t = case["tokens"]
        x = torch.randn(t, case["heads"] + case["rest"], d, generator=gen, device="cuda").to(dtype)
        if t == 1:
            pos = torch.randint(0, case["top"] + 1, (1,), generator=gen, device="cuda")
        else:                                                   # the end of a text of `top` + 1 tokens
            pos = (torch.arange(t, device="cuda") + max(0, case["top"] + 1 - t))
        return dict(x=x, pos=pos)
    if case["op"] == "append":
        new, old = _ints(case, "new"), _ints(case, "old")
        lens = [a + b for a, b in zip(new, old)]
    else:
        lens = _ints(case, "kv_lens")
    table, n_pages = _page_table(gen, lens, case["page"])
    k, v = _kv(gen, sum(lens), case["hkv"], d, dtype)
    i = dict(k=k, v=v, table=table, n_pages=n_pages, lens=lens)
    if case["op"] != "append":
        n_q = sum(_ints(case, "q_lens"))
        i["q"] = (1.5 * torch.randn(n_q, case["hq"], d, generator=gen, device="cuda")).to(dtype)
    return i


SCALING = {"none": {}, "linear": dict(factor=4.0), "wavelength": dict(factor=8.0, original_length=8192, low=1.0, high=4.0),
           "yarn": dict(factor=16.0, original_length=4096, low=1.0, high=32.0)}


def prepare(case, seed):
    i = _inputs(case, seed)
    s = dict(case=case)
    if own:
        from w4a16_dequant_gemm_group_amd import binding as B
    if case["op"] == "rope":
        s.update(x=i["x"], pos=i["pos"])
        if own:
            s["freqs"], s["amplitude"] = B.gq_rope_frequencies(case["rot"], 500000.0, case["scaling"],
                                                               **SCALING[case["scaling"]], device="cuda")
        else:
            s["freqs"], s["amplitude"] = _plain_frequencies(case["rot"], case["scaling"])
        return s
    dtype, h, d, page = DTYPES[case["dtype"]], case["hkv"], case["d"], case["page"]
    dev32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    with_bounds = case["op"] != "attention"
    if own:
        s["cache"] = B.gq_kv8_empty(i["n_pages"], h, d, page, device="cuda")
        s["bounds"] = B.gq_kv8_bounds_empty(i["n_pages"], h, d, dtype, device="cuda").zero_() if with_bounds else None
    else:
        s["cache"] = _plain_empty(i["n_pages"], h, d, page)
        s["bounds"] = torch.zeros(i["n_pages"], h, 2, d, dtype=dtype, device="cuda") if with_bounds else None
    s["table"] = i["table"]
    if case["op"] == "append":
        new, old = _ints(case, "new"), _ints(case, "old")
        # what is there already enters in a call of its own, the rest is what `run` appends
        first, rest, at = [], [], 0
        for m, o in zip(new, old):
            first.append(torch.arange(at, at + o, device="cuda"))
            rest.append(torch.arange(at + o, at + o + m, device="cuda"))
            at += o + m
        first, rest = torch.cat(first), torch.cat(rest)
        s.update(old=old, new=new, k=i["k"][rest], v=i["v"][rest], lens=dev32(i["lens"]), starts=dev32(_starts(new)),
                 slots=_touched_slots(case, i["table"]))
        k, v, lens = i["k"][first], i["v"][first], old
    else:
        k, v, lens = i["k"], i["v"], i["lens"]
        q_lens = _ints(case, "q_lens")
        s.update(q=i["q"], q_lens=q_lens, kv_lens=lens, starts=dev32(_starts(q_lens)), lens=dev32(lens))
    if sum(lens):
        if own:
            B.gq_kv8_append(k, v, s["cache"], s["table"], dev32(lens), starts=dev32(_starts(lens)), bounds=s["bounds"])
        else:
            _plain_append(k, v, s["cache"], s["table"], [0] * len(lens), lens, s["bounds"], page)
    return s


def _touched_slots(case, table):
    """Slots of the tokens in the blocks that an append touches, older ones among them."""
    page, out = case["page"], []
    for b, (m, o) in enumerate(zip(_ints(case, "new"), _ints(case, "old"))):
        pos = torch.arange(o // BLOCK * BLOCK, o + m, device="cuda")
        out.append(table[b].long()[pos // page] * page + pos % page)
    return torch.cat(out)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from w4a16_dequant_gemm_group_amd import binding as B
        if op == "rope":
            return B.gq_rope(state["x"][:, :c["heads"]], state["pos"], state["freqs"], interleaved=c["interleaved"],
                             amplitude=state["amplitude"], inverse=c["inverse"])
        cache, table, lens = state["cache"], state["table"], state["lens"]
        if op == "append":
            single = max(state["new"]) == 1
            B.gq_kv8_append(state["k"], state["v"], cache, table, lens, starts=None if single else state["starts"],
                            bounds=state["bounds"])
            k, v = B.gq_kv8_read(cache, state["slots"], c["d"], out_dtype=DTYPES[c["dtype"]])
            return k, v, state["bounds"]
        single = max(state["q_lens"]) == 1
        starts = None if single else state["starts"]
        if op == "attention":
            return B.gq_kv8_attention(state["q"], cache, table, lens, q_starts=starts, max_q_len=max(state["q_lens"]),
                                      max_kv_len=max(state["kv_lens"]), causal=True, window=c["window"],
                                      return_lse=c["lse"])
        pages, seen = B.gq_kv8_select(state["q"], state["bounds"], table, lens, c["keep"], c["page"], q_starts=starts,
                                      max_kv_len=max(state["kv_lens"]), first=c["first"], last=c["last"])
        out = B.gq_kv8_attention(state["q"], cache, pages, seen)
        return pages, seen, out
    if op == "rope":
        return _plain_rope(state)
    if op == "append":
        _plain_append(state["k"], state["v"], state["cache"], state["table"], state["old"], state["new"],
                      state["bounds"], c["page"])
        k, v = _plain_read(state["cache"], state["slots"])
        return k.to(DTYPES[c["dtype"]]), v.to(DTYPES[c["dtype"]]), state["bounds"]
    return _plain_attention(state) if op == "attention" else _plain_sparse(state)


def _plain_frequencies(rot, scaling):
    """Angles per position (64 bits) of the rot / 2 pairs, and the factor of the result."""
    base, p = 500000.0, SCALING[scaling]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = torch.exp(-2.0 * i / rot * math.log(base))
    if scaling == "none":
        return f, 1.0
    s = p["factor"]
    if scaling == "linear":
        return f / s, 1.0
    if scaling == "wavelength":
        turns = p["original_length"] * f / (2 * math.pi)
        t = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        return (1 - t) * f / s + t * f, 1.0
    dim = lambda turns: rot * math.log(p["original_length"] / (2 * math.pi * turns)) / (2 * math.log(base))
    lo = max(math.floor(dim(p["high"])), 0)
    hi = max(min(math.ceil(dim(p["low"])), rot - 1), lo + 0.001)
    t = 1 - ((i - lo) / (hi - lo)).clamp(0, 1)
    return (1 - t) * f / s + t * f, 0.1 * math.log(s) + 1.0


def _plain_rope(state):
    c = state["case"]
    rot = c["rot"]
    x = state["x"][:, :c["heads"]].float()
    a = (state["pos"].double()[:, None] * state["freqs"])[:, None]
    cos, sin = (a.cos() * state["amplitude"]).float(), (a.sin() * state["amplitude"]).float()
    if c["inverse"]:
        sin = -sin
    y = x.clone()
    if c["interleaved"]:
        p, q = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = p * cos - q * sin
        y[..., 1:rot:2] = q * cos + p * sin
    else:
        p, q = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = p * cos - q * sin
        y[..., rot // 2:rot] = q * cos + p * sin
    return y.to(state["x"].dtype)


def _plain_empty(n_pages, h, d, page):
    out = {}
    for x in "kv":
        out[x] = torch.zeros(n_pages * page, h, d, dtype=torch.int8, device="cuda")
        out[x + "s"] = torch.zeros(n_pages * page // BLOCK, h, dtype=torch.float32, device="cuda")
    return out


def _plain_append(k, v, cache, table, old, new, bounds, page):
    """Tokens of all sequences, packed, behind old[b] tokens each.  Codes in 64 bits:
    they are roundings, and a value next to a border must fall on the right side."""
    dev = k.device
    seq = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev), output_size=sum(new))
    first = torch.tensor(_starts(new)[:-1], device=dev)
    base = torch.tensor(old, device=dev)
    pos = torch.arange(sum(new), device=dev) - first[seq] + base[seq]
    slot = table[seq, pos // page].long() * page + pos % page
    block = slot // BLOCK
    # tokens of earlier calls in the block that a sequence's first new token enters
    some = torch.tensor([b for b, (m, o) in enumerate(zip(new, old)) if m and o % BLOCK], dtype=torch.long, device=dev)
    place = torch.arange(BLOCK, device=dev)
    opos = base[some, None] // BLOCK * BLOCK + place
    oslot = table[some[:, None], opos // page].long() * page + opos % page
    oblock = oslot[:, 0] // BLOCK
    oslot = oslot[opos < base[some, None]]
    for name, x in (("k", k), ("v", v)):
        codes, scales = cache[name], cache[name + "s"]
        s = torch.zeros_like(scales)
        s.scatter_reduce_(0, block[:, None].expand(-1, x.shape[1]), (x.abs().amax(-1).double() / 127.0).float(), "amax")
        s = s.clamp(min=LEAST)
        before = scales[oblock]
        s[oblock] = torch.maximum(s[oblock], before)
        if oslot.numel():
            ratio = torch.zeros_like(scales, dtype=torch.float64)
            ratio[oblock] = before.double()
            b = oslot // BLOCK
            codes[oslot] = torch.round(codes[oslot].double() * ratio[b][..., None] / s[b].double()[..., None]).to(torch.int8)
        codes[slot] = torch.round(x.double() / s[block].double()[..., None]).clamp(-127, 127).to(torch.int8)
        scales[block] = s[block]
    if bounds is not None:
        inf = float("inf")
        pg = slot // page
        at = pg[:, None, None].expand(-1, *k.shape[1:])
        n_pages = bounds.shape[0]
        lo = torch.full((n_pages, *k.shape[1:]), inf, dtype=torch.float32, device=dev).scatter_reduce_(0, at, k.float(), "amin")
        hi = torch.full((n_pages, *k.shape[1:]), -inf, dtype=torch.float32, device=dev).scatter_reduce_(0, at, k.float(), "amax")
        kept = torch.tensor([b for b, (m, o) in enumerate(zip(new, old)) if m and o % page], dtype=torch.long, device=dev)
        opage = table[kept, base[kept] // page].long()
        lo[opage] = torch.minimum(lo[opage], bounds[opage, :, 0].float())
        hi[opage] = torch.maximum(hi[opage], bounds[opage, :, 1].float())
        bounds[pg, :, 0] = lo[pg].to(bounds.dtype)
        bounds[pg, :, 1] = hi[pg].to(bounds.dtype)


def _plain_read(cache, slots):
    """Values of the given slots in float32."""
    return [cache[x][slots].float() * cache[x + "s"][slots // BLOCK][..., None] for x in "kv"]


def _plain_rows(q, k, v, r, hide):
    """q [hkv, r * n, d] scaled, k and v [kv, hkv, d], hide [n, kv] or [hkv, n, kv] -> o, lse [hkv, r, n, ...]."""
    hkv, rows, d = q.shape
    s = torch.matmul(q, k.permute(1, 2, 0).contiguous()).view(hkv, r, rows // r, -1)
    s = s.masked_fill(hide, float("-inf"))
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul((e / l).view(hkv, rows, -1), v.transpose(0, 1).contiguous())
    return o.view(hkv, r, rows // r, d), (m + torch.log(l)).view(hkv, r, rows // r)


def _plain_attention(state):
    c = state["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    r = hq // hkv
    q = state["q"].float() * (1.0 / math.sqrt(d))
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    at = 0
    for b, (n, kv) in enumerate(zip(state["q_lens"], state["kv_lens"])):
        t0 = max(0, kv - n - c["window"] + 1) if c["window"] else 0   # a window's earliest key
        pos = torch.arange(t0, kv, device="cuda")
        k, v = _plain_read(state["cache"], state["table"][b].long()[pos // page] * page + pos % page)
        qb = q[at:at + n].view(n, hkv, r, d).permute(1, 2, 0, 3).reshape(hkv, r * n, d)
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        hide = pos > p
        if c["window"]:
            hide = hide | (pos <= p - c["window"])
        o, s = _plain_rows(qb, k, v, r, hide)
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, hq, d)
        lse[at:at + n] = s.permute(2, 0, 1).reshape(n, hq)
        at += n
    out = out.to(state["q"].dtype)
    return (out, lse) if c["lse"] else out


def _plain_sparse(state):
    c = state["case"]
    hq, hkv, d, page, keep = c["hq"], c["hkv"], c["d"], c["page"], c["keep"]
    r = hq // hkv
    q = state["q"]
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    pages = torch.full((q.shape[0], hkv, keep), -1, dtype=torch.int32, device="cuda")
    lens = torch.empty(q.shape[0], dtype=torch.int32, device="cuda")
    at = 0
    for b, (n, kv) in enumerate(zip(state["q_lens"], state["kv_lens"])):
        row = state["table"][b].long()
        for p in range(kv - n, kv):
            n_all = p // page + 1
            qh = q[at].view(hkv, r, d)
            # scores in 64 bits: the choice turns on their order
            bd = state["bounds"][row[:n_all]].double()                        # [pages, hkv, 2, d]
            qd = qh.double()
            score = torch.matmul(qd.clamp(min=0), bd[:, :, 1].permute(1, 2, 0).contiguous()) + \
                torch.matmul(qd.clamp(max=0), bd[:, :, 0].permute(1, 2, 0).contiguous())
            score = score.amax(1)                                             # [hkv, pages]
            j = torch.arange(n_all, device="cuda")
            score = score.masked_fill((j < c["first"]) | (j >= n_all - c["last"]), float("inf"))
            n_sel = min(keep, n_all)
            chosen = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :n_sel]
            chosen = torch.sort(chosen, dim=-1).values                        # [hkv, n_sel]
            pages[at, :, :n_sel] = row[chosen].to(torch.int32)
            seen = (n_sel - 1) * page + p % page + 1
            lens[at] = seen
            slots = (row[chosen] * page)[..., None] + torch.arange(page, device="cuda")
            slots = slots.view(hkv, -1)[:, :seen]                             # [hkv, seen]
            head = torch.arange(hkv, device="cuda")[:, None]
            kv_of = [state["cache"][x][slots, head].float() * state["cache"][x + "s"][slots // BLOCK, head][..., None]
                     for x in "kv"]                                           # [hkv, seen, d]
            s = torch.matmul(qh.float() * (1.0 / math.sqrt(d)), kv_of[0].transpose(1, 2).contiguous())
            e = torch.exp(s - s.amax(-1, keepdim=True))
            out[at] = torch.matmul(e / e.sum(-1, keepdim=True), kv_of[1]).reshape(hq, d)
            at += 1
    return pages, lens, out.to(q.dtype)


# ---------------------------------------------------------------------------
# The definition, in 64 bits
# ---------------------------------------------------------------------------

def _exact_angles(case):
    rot, kind, p = case["rot"], case["scaling"], SCALING[case["scaling"]]
    f = [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    m = 1.0
    if kind == "linear":
        f = [x / p["factor"] for x in f]
    elif kind == "wavelength":
        for i, x in enumerate(f):
            length = 2 * math.pi / x
            if length > p["original_length"] / p["low"]:
                f[i] = x / p["factor"]
            elif length > p["original_length"] / p["high"]:
                t = (p["original_length"] / length - p["low"]) / (p["high"] - p["low"])
                f[i] = (1 - t) * x / p["factor"] + t * x
    elif kind == "yarn":
        at = [rot * math.log(p["original_length"] / (2 * math.pi * b)) / (2 * math.log(500000.0)) for b in (p["high"], p["low"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        hi = max(hi, lo + 0.001)
        for i, x in enumerate(f):
            t = min(max((i - lo) / (hi - lo), 0.0), 1.0)               # 0: as it is, 1: stretched
            f[i] = x * (1 - t) + x / p["factor"] * t
        m = 0.1 * math.log(p["factor"]) + 1.0
    return torch.tensor(f, dtype=torch.float64, device="cuda"), m


def _exact_blocks(x, old):
    """One sequence's x [n, h, d], of which the first `old` tokens came in an earlier
    call: the values that the blocks of 16 stand for."""
    n, h, d = x.shape
    pad = -n % BLOCK
    b = torch.cat([x.double(), x.new_zeros(pad, h, d).double()]).view(-1, BLOCK, h, d)
    early = (torch.arange(n + pad, device=x.device) < old).view(-1, BLOCK, 1, 1)

    def scale(y):
        s = y.abs().amax((1, 3), keepdim=True) / 127
        return s.to(torch.float32).double().clamp(min=LEAST)
    s0 = scale(b * early)
    s1 = torch.maximum(torch.where(early.any(1, keepdim=True), s0, 0.0), scale(b * ~early))
    # blocks that the later call does not touch keep their scale
    s1 = torch.where(early.all(1, keepdim=True), s0, s1)
    codes = torch.where(early, torch.round(torch.round(b / s0) * s0 / s1), torch.round(b / s1)).clamp(-127, 127)
    return (codes * s1).view(-1, h, d)[:n]


def exact(case, seed):
    i = _inputs(case, seed)
    if case["op"] == "rope":
        f, m = _exact_angles(case)
        rot = case["rot"]
        x = i["x"][:, :case["heads"]].double()
        a = i["pos"].double()[:, None, None] * f * (-1.0 if case["inverse"] else 1.0)
        turn = torch.polar(torch.full_like(a, m), a)
        part = x[..., :rot]
        pair = part.reshape(*part.shape[:-1], rot // 2, 2) if case["interleaved"] else \
            part.reshape(*part.shape[:-1], 2, rot // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat((z.reshape(part.shape), x[..., rot:]), -1)
    page, h, d = case["page"], case["hkv"], case["d"]
    lens, at = i["lens"], 0
    old = _ints(case, "old") if case["op"] == "append" else [0] * len(lens)
    ks, vs = [], []
    for n, o in zip(lens, old):
        ks.append(_exact_blocks(i["k"][at:at + n], o))
        vs.append(_exact_blocks(i["v"][at:at + n], o))
        at += n
    bounds = torch.zeros(i["n_pages"], h, 2, d, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            part = i["k"][at + j * page:at + min(n, (j + 1) * page)].double()
            bounds[i["table"][b, j], :, 0] = part.amin(0)
            bounds[i["table"][b, j], :, 1] = part.amax(0)
        at += n
    if case["op"] == "append":
        cut = [o // BLOCK * BLOCK for o in old]
        return torch.cat([x[c:] for x, c in zip(ks, cut)]), torch.cat([x[c:] for x, c in zip(vs, cut)]), bounds
    hq, rep = case["hq"], case["hq"] // h
    q_lens = _ints(case, "q_lens")
    q = i["q"].double()
    out = torch.zeros(sum(q_lens), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(q_lens), hq, dtype=torch.float64, device="cuda")
    if case["op"] == "sparse":
        pages = torch.full((sum(q_lens), h, case["keep"]), -1, dtype=torch.int32, device="cuda")
        seen = torch.zeros(sum(q_lens), dtype=torch.int32, device="cuda")
    qa = 0
    for b, (n, kv) in enumerate(zip(q_lens, lens)):
        k, v = ks[b], vs[b]
        if case["op"] == "attention":
            w = case["window"]
            for a in range(0, n, 1024):                              # query blocks bound the memory
                e = min(n, a + 1024)
                last = kv - n + e                                    # keys 0 .. last - 1 can be seen
                i_pos = torch.arange(kv - n + a, last, device="cuda").unsqueeze(1)
                j_pos = torch.arange(last, device="cuda").unsqueeze(0)
                ok = j_pos <= i_pos
                if w:
                    ok &= j_pos > i_pos - w
                for x in range(hq):
                    logits = q[qa + a:qa + e, x] @ k[:last, x // rep].T.contiguous()
                    logits = torch.where(ok, logits / d ** 0.5, -math.inf)
                    norm = torch.logsumexp(logits, 1)
                    out[qa + a:qa + e, x] = torch.exp(logits - norm[:, None]) @ v[:last, x // rep]
                    lse[qa + a:qa + e, x] = norm
        else:
            for t in range(n):
                p = kv - n + t
                n_all = p // page + 1
                take = min(case["keep"], n_all)
                seen[qa + t] = (take - 1) * page + p % page + 1
                bd = bounds[i["table"][b, :n_all].long()]             # [pages, h, 2, d]
                for x in range(h):
                    best = None
                    for y in range(x * rep, (x + 1) * rep):
                        top = torch.maximum(q[qa + t, y] * bd[:, x, 0], q[qa + t, y] * bd[:, x, 1]).sum(-1)
                        best = top if best is None else torch.maximum(best, top)
                    best = best.cpu().tolist()
                    always = [j for j in range(n_all) if j < case["first"] or j >= n_all - case["last"]]
                    order = always + sorted(set(range(n_all)) - set(always), key=lambda j: (-best[j], j))
                    mine = sorted(order[:take])
                    pages[qa + t, x, :take] = i["table"][b, mine]
                    pos = torch.cat([torch.arange(j * page, min((j + 1) * page, p + 1), device="cuda") for j in mine])
                    for y in range(x * rep, (x + 1) * rep):
                        w = torch.softmax(k[pos, x] @ q[qa + t, y] / d ** 0.5, 0)
                        out[qa + t, y] = w @ v[pos, x]
        qa += n
    if case["op"] == "sparse":
        return pages, seen, out
    return (out, lse) if case["lse"] else out
