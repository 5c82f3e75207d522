"""Cases of the serving-step operators: page plan, rotary tables, norm + rotation + append, and
attention of one or a few new tokens over the packed cache.

``run`` makes one pass through one operator, either in its plain form (elementary torch operations)
or, where ``own`` is set, through the library's entry points.  ``prepare`` holds what a serving
program has in hand before the call.  Layouts and formulas are those of include/lkv.h.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 256  # tokens of a page


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a small batch: 16 requests near 8k tokens, one new token each (latency)
        {"name": "plan_decode_16", "op": "plan", "B": 16, "pps": 33, "lo": 7900, "hi": 8192, "new_lo": 1, "new_hi": 1},
        # a large mixed batch: decodes and prompts, a hundred thousand new tokens
        {"name": "plan_mixed_777", "op": "plan", "B": 777, "pps": 40, "lo": 0, "hi": 8000, "new_lo": 1, "new_hi": 1500},
        # the tables of an 8k-token model, frequencies blended by wavelength
        {"name": "table_8192", "op": "table", "rot": 128, "rows": 8192, "kind": "smooth", "base": 500000.0, "factor": 8.0},
        # a long-context table, ramp over the dimensions, odd number of rows, part of a head
        {"name": "table_131071", "op": "table", "rot": 96, "rows": 131071, "kind": "ramp", "base": 10000.0, "factor": 32.0},
        # the new token of 16 requests: 32 query / 8 KV heads, K6V4 in groups of 64, paged (latency)
        {"name": "append_decode_16", "op": "append", "N": 16, "cap": 16, "Hq": 32, "Hkv": 8, "D": 128, "kb": 6, "vb": 4,
         "G": 64, "rot": 128, "inter": False, "norm": True, "seqs": 16, "paged": True, "max_pos": 8192},
        # a padded ragged batch, heads of 64 with a quarter rotated in pairs, 8-bit cache, contiguous
        {"name": "append_padded_777", "op": "append", "N": 777, "cap": 1024, "Hq": 12, "Hkv": 3, "D": 64, "kb": 8,
         "vb": 8, "G": 32, "rot": 16, "inter": True, "norm": False, "seqs": 7, "paged": False, "max_pos": 4096},
        # prompts of 16k tokens in all, entering the paged K6V4 cache
        {"name": "append_prompts_16384", "op": "append", "N": 16384, "cap": 16384, "Hq": 32, "Hkv": 8, "D": 128, "kb": 6,
         "vb": 4, "G": 64, "rot": 128, "inter": False, "norm": True, "seqs": 5, "paged": True, "max_pos": 32768},
        # the tiny decode of the tests: 4 query / 2 KV heads of 64, 256 tokens, capped scores (latency)
        {"name": "attend_tiny_256", "op": "attend", "B": 1, "Hq": 4, "Hkv": 2, "D": 64, "G": 32, "kb": 6, "vb": 4,
         "lo": 256, "hi": 256, "nq": 1, "paged": False, "cap": 30.0, "bias": False, "window": 0, "prefix": 0, "docs": False},
        # the Llama-3.1-8B-shaped decode step over a paged cache, with capped scores
        {"name": "attend_paged_8192", "op": "attend", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "G": 64, "kb": 6, "vb": 4,
         "lo": 8192, "hi": 8192, "nq": 1, "paged": True, "cap": 50.0, "bias": False, "window": 0, "prefix": 0, "docs": False},
        # four drafted tokens verified against one long context, scores biased by distance
        {"name": "attend_verify_131072", "op": "attend", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "G": 64, "kb": 6, "vb": 4,
         "lo": 131072, "hi": 131072, "nq": 4, "paged": False, "cap": 0.0, "bias": True, "window": 0, "prefix": 0, "docs": False},
        # a ragged batch of 64 with an 8-bit cache, a window of 1024 and a prefix that stays visible
        {"name": "attend_window_64", "op": "attend", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "G": 32, "kb": 8, "vb": 8,
         "lo": 512, "hi": 4096, "nq": 1, "paged": True, "cap": 0.0, "bias": False, "window": 1024, "prefix": 37, "docs": False},
        # runs of up to 8 drafted tokens, groups of 8 query heads, 16-bit outlier layer, packed documents
        {"name": "attend_docs_16bit", "op": "attend", "B": 9, "Hq": 32, "Hkv": 4, "D": 128, "G": 64, "kb": 16, "vb": 16,
         "lo": 1001, "hi": 9001, "nq": 8, "paged": False, "cap": 0.0, "bias": False, "window": 0, "prefix": 0, "docs": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "table", "append", "append", "attend", "attend", "attend"])
    if op == "plan":
        B = _log(rng, 1, 1000)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(3000, 200000 // B)))
        return {"op": "plan", "B": B, "pps": rng.randint(44, 60), "lo": 0, "hi": _log(rng, 100, 8192), "new_lo": min(1, new), "new_hi": new}
    if op == "table":
        return {"op": "table", "rot": 16 * rng.randint(1, 8), "rows": _log(rng, 257, 131071),
                "kind": rng.choice(["none", "linear", "smooth", "ramp"]), "base": rng.choice([10000.0, 500000.0]),
                "factor": rng.choice([2.0, 8.0, 32.0])}
    D = rng.choice([64, 128])
    G = rng.choice([g for g in (32, 64, 128) if g <= D])
    kb, vb = rng.choice([(6, 4), (6, 4), (8, 8), (4, 4), (4, 2), (6, 6), (16, 16), (16, 4)])
    if op == "append":
        N = _log(rng, 1, 12000)
        Hkv = rng.choice([1, 2, 3, 8])
        return {"op": "append", "N": N, "cap": N + rng.choice([0, 0, 5, 64]), "Hq": Hkv * rng.choice([1, 2, 4]), "Hkv": Hkv, "D": D,
                "kb": kb, "vb": vb, "G": G, "rot": 16 * rng.randint(0, D // 16), "inter": rng.random() < 0.5,
                "norm": rng.random() < 0.6, "seqs": rng.randint(1, min(N, 40)), "paged": rng.random() < 0.6, "max_pos": 16384}
    B, Hkv, r = _log(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    bits = kb + vb
    top = max(300, min(100000, int(1.2e9 / (B * Hkv * D * bits))))
    hi = _log(rng, 257, top)
    nq = rng.choice([1, 1, 1, 2, 3, 5, 8])
    return {"op": "attend", "B": B, "Hq": Hkv * r, "Hkv": Hkv, "D": D, "G": G, "kb": kb, "vb": vb, "lo": max(nq, hi // rng.randint(1, 9)),
            "hi": hi, "nq": nq, "paged": rng.random() < 0.5, "cap": rng.choice([0.0, 0.0, 30.0, 50.0]), "bias": rng.random() < 0.3,
            "window": rng.choice([0, 0, _log(rng, 1, 4096)]), "prefix": rng.choice([0, 0, _log(rng, 1, 300)]), "docs": rng.random() < 0.25}


# ------------------------------------------------------------------ what a case fixes whatever the seed
def _fixed(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _ints(rng, lo, hi, n):
    return [rng.randint(lo, hi) for _ in range(n)]


def _plan_lens(c):
    rng = _fixed(c)
    return _ints(rng, c["lo"], c["hi"], c["B"]), _ints(rng, c["new_lo"], c["new_hi"], c["B"])


def _attend_lens(c):
    """Cached tokens, new tokens, prefix and document start of each sequence."""
    rng = _fixed(c)
    lens = _ints(rng, c["lo"], c["hi"], c["B"])
    n = [c["nq"]] * c["B"] if c["nq"] <= 4 else [min(t, rng.randint(1, c["nq"])) for t in lens]
    prefix = [min(t, c["prefix"]) for t in lens]
    start = [rng.randint(0, t // 2) if c["docs"] else 0 for t in lens]
    return lens, n, prefix, start


def _visible(c):
    """(rows read, (query, row) pairs) of one KV head over all sequences."""
    rows = pairs = 0
    for T, n, pre, st in zip(*_attend_lens(c)):
        low = max(st, T - n - c["window"] + 1 if c["window"] else 0, 0)
        rows += min(pre, low) + T - low
        for i in range(n):
            p = T - n + i
            lo_i = max(st, p - c["window"] + 1 if c["window"] else 0)
            pairs += max(0, p + 1 - max(lo_i, min(pre, p + 1))) + min(pre, T)
    return rows, pairs


def _row_bytes(bits, D, G):
    return D * bits // 8 + (0 if bits == 16 else 8 * (D // G))


def work(case):
    c = case
    if c["op"] == "plan":
        lens, new = _plan_lens(c)
        pages = sum((t + n + PAGE - 1) // PAGE - (t + PAGE - 1) // PAGE for t, n in zip(lens, new))
        tokens = sum(new)
        return {"bytes": 8 * c["B"] + 8 * pages + 16 * tokens + 8 * c["B"] + 4 * pages + 16, "flops": 0}
    if c["op"] == "table":
        return {"bytes": c["rows"] * c["rot"] * 4, "flops": 4 * c["rows"] * c["rot"]}
    if c["op"] == "append":
        D, G = c["D"], c["G"]
        token = 2 * D * (2 * c["Hq"] + 2 * c["Hkv"]) + c["Hkv"] * (_row_bytes(c["kb"], D, G) + _row_bytes(c["vb"], D, G)) + 4 * c["rot"] + 12
        return {"bytes": c["N"] * token, "flops": c["N"] * D * (c["Hq"] + c["Hkv"]) * 8}
    rows, pairs = _visible(c)
    n = sum(_attend_lens(c)[1])
    kv = rows * c["Hkv"] * (_row_bytes(c["kb"], c["D"], c["G"]) + _row_bytes(c["vb"], c["D"], c["G"]))
    return {"bytes": kv + n * c["Hq"] * (c["D"] * 6 + 4), "flops": 4 * c["D"] * c["Hq"] * pairs}


# ------------------------------------------------------------------ inputs
def _quantized(x, bits, G):
    """Codes (int64 [..., D]) and (scale, zero) of bf16 values held in f32, in the library's fixed fp32 formula."""
    g = x.unflatten(-1, (-1, G))
    mn, mx = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    d, qmax = mx - mn, float(2 ** bits - 1)
    flat = d == 0
    scale = torch.where(flat, 0.0, d / qmax)
    inv = torch.where(flat, 0.0, qmax / torch.where(flat, 1.0, d))
    codes = torch.round((g - mn) * inv).clamp(0, qmax).to(torch.int64)
    return codes.flatten(-2), torch.cat([scale, mn + 0.0], -1)


def _packed(codes, bits):
    """Codes of a row as one little-endian bit string: 8 codes fill `bits` bytes."""
    if bits == 8:
        return codes.to(torch.uint8)
    at = torch.arange(8, device=codes.device)
    word = (codes.unflatten(-1, (-1, 8)) << (at * bits)).sum(-1, keepdim=True)
    return ((word >> (at[:bits] * 8)) & 255).to(torch.uint8).flatten(-2)


def _rows(x, bits, G):
    """(codes u8 [..., D * bits / 8], sz f32 [..., D / G, 2] or None) of bf16 rows."""
    if bits == 16:
        return x.contiguous().view(torch.uint8), None
    codes, sz = _quantized(x.float(), bits, G)
    return _packed(codes, bits), sz


def _values(codes, sz, bits, D):
    """The f32 values that packed rows stand for."""
    if bits == 16:
        return codes.contiguous().view(torch.bfloat16).float()
    at = torch.arange(8, device=codes.device)
    word = (codes.unflatten(-1, (-1, bits)).to(torch.int64) << (at[:bits] * 8)).sum(-1, keepdim=True)
    c = ((word >> (at * bits)) & (2 ** bits - 1)).flatten(-2).float()
    c = c.unflatten(-1, (sz.shape[-2], -1))
    return (c * sz[..., 0:1] + sz[..., 1:2]).flatten(-2)


def _channel_scales(gen, Hkv, D):
    """K's channel scales: log-uniform in [0.5, 4], two outlier channels of each head 15 times larger."""
    s = torch.exp(math.log(0.5) + torch.rand(Hkv, D, generator=gen, device="cuda") * math.log(8.0))
    return s * torch.where(torch.rand(Hkv, D, generator=gen, device="cuda").argsort(-1) < 2, 15.0, 1.0)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_plan(c, gen, seed):
    lens, new = _plan_lens(c)
    old = [(t + PAGE - 1) // PAGE for t in lens]
    need = sum((t + n + PAGE - 1) // PAGE - o for t, n, o in zip(lens, new, old))
    used = sum(old)
    pages = used + need + 7
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor(np.cumsum([0] + old[:-1]), device="cuda")
    at = torch.arange(c["pps"], device="cuda")
    table = torch.where(at < _i32(old)[:, None], perm[(first[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32)
    cap = sum(new) + 3
    return {"lens": _i32(lens), "new": _i32(new), "table": table, "pages": pages, "free": perm[used:].contiguous(),
            "free_count": _i32([pages - used]), "cap": cap, "new_lens": torch.full_like(_i32(lens), -1),
            "cu": torch.full((c["B"] + 1,), -1, dtype=torch.int32, device="cuda"),
            "pos": torch.full((cap,), -1, dtype=torch.int32, device="cuda"),
            "seq": torch.full((cap,), -1, dtype=torch.int32, device="cuda"),
            "slots": torch.full((cap,), -1, dtype=torch.int64, device="cuda"),
            "left": _i32([-1]), "status": _i32([-1])}


def _prepare_append(c, gen, seed):
    D, Hq, Hkv, N, cap = c["D"], c["Hq"], c["Hkv"], c["N"], c["cap"]
    x = torch.randn(cap, Hq + 2 * Hkv, D, generator=gen, device="cuda")
    x[:, Hq:Hq + Hkv] *= _channel_scales(gen, Hkv, D)
    x = x.to(torch.bfloat16)
    weights = (1.0 + 0.2 * torch.randn(2, D, generator=gen, device="cuda")).to(torch.bfloat16)
    # the tokens of `seqs` sequences, each a run of positions behind what is cached already
    rng = _fixed(c)
    cuts = sorted(rng.sample(range(1, N), c["seqs"] - 1)) if c["seqs"] > 1 else []
    runs = [b - a for a, b in zip([0] + cuts, cuts + [N])]
    begins = [rng.randint(0, max(0, c["max_pos"] - n)) if n < c["max_pos"] else 0 for n in runs]
    owner = torch.repeat_interleave(torch.arange(len(runs), device="cuda"), torch.tensor(runs, device="cuda"), output_size=N)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(begins, runs)]).cuda()
    if c["paged"]:
        used = [(a // PAGE, (a + n - 1) // PAGE) for a, n in zip(begins, runs)]
        many = [b - a + 1 for a, b in used]
        perm = torch.randperm(sum(many), generator=gen, device="cuda")
        first = torch.tensor([sum(many[:i]) - used[i][0] for i in range(len(many))], device="cuda")
        slots = perm[first[owner] + pos // PAGE] * PAGE + pos % PAGE
        pages, page_tokens = sum(many) + 1, PAGE
    else:
        page_tokens = max(a + n for a, n in zip(begins, runs)) // 2 * 2 + 2
        slots, pages = owner * page_tokens + pos, c["seqs"] + 1
    pad = torch.zeros(cap - N, dtype=torch.int64, device="cuda")
    mk = lambda b: torch.zeros(pages, Hkv, page_tokens, D * b // 8, dtype=torch.uint8, device="cuda")  # noqa: E731
    sz = lambda b: None if b == 16 else torch.zeros(pages, Hkv, page_tokens, D // c["G"], 2, device="cuda")  # noqa: E731
    f = c["base"] if "base" in c else 10000.0
    half = max(c["rot"] // 2, 1)
    angle = torch.arange(c["max_pos"], device="cuda", dtype=torch.float64)[:, None] * f ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    return {"x": x, "q": x[:, :Hq], "k": x[:, Hq:Hq + Hkv], "v": x[:, Hq + Hkv:], "weights": weights, "eps": 1e-6,
            "pos": torch.cat([pos, pad]).to(torch.int32), "slots": torch.cat([slots, pad - 1]), "count": _i32([N]),
            "table": torch.stack([angle.cos(), angle.sin()], -1).float(), "pages": pages, "page_tokens": page_tokens,
            "q_out": torch.zeros(cap, Hq, D, dtype=torch.bfloat16, device="cuda"),
            "k_codes": mk(c["kb"]), "k_sz": sz(c["kb"]), "v_codes": mk(c["vb"]), "v_sz": sz(c["vb"])}


def _prepare_attend(c, gen, seed):
    B, Hq, Hkv, D, G = c["B"], c["Hq"], c["Hkv"], c["D"], c["G"]
    lens, n, prefix, start = _attend_lens(c)
    pps = (max(lens) + PAGE - 1) // PAGE
    T = pps * PAGE if c["paged"] else max(lens) + max(lens) % 2
    N, r = sum(n), Hq // Hkv
    q = torch.randn(N, Hq, D, generator=gen, device="cuda").to(torch.bfloat16)
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda")
    k = torch.randn(B, Hkv, T, D, generator=gen, device="cuda") * _channel_scales(gen, Hkv, D)[:, None]
    # heavy hitters: one token in 500 lies along the group's mean query and makes the softmax peaky
    mean = q[cu[:-1].long()].float().view(B, Hkv, r, D).mean(2)
    heavy = torch.rand(B, 1, T, 1, generator=gen, device="cuda") < 0.002
    k = torch.where(heavy, 4.0 * mean[:, :, None] + torch.randn(B, Hkv, T, D, generator=gen, device="cuda"), k).to(torch.bfloat16)
    v = torch.randn(B, Hkv, T, D, generator=gen, device="cuda").to(torch.bfloat16)
    s = {"q": q, "cu": cu, "lens": _i32(lens), "T": T, "pps": pps, "pages": B * pps + 3, "N": N, "max_q": max(n), "table": None,
         "prefix": _i32(prefix) if c["prefix"] else None, "start": _i32(start) if c["docs"] else None,
         "slopes": torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float() if c["bias"] else None,
         "scale": D ** -0.5, "out": torch.zeros(N, Hq, D, device="cuda"), "lse": torch.zeros(N, Hq, device="cuda")}
    for key, x, bits in (("k", k, c["kb"]), ("v", v, c["vb"])):
        s[key + "_codes"], s[key + "_sz"] = _rows(x, bits, G)
    if c["paged"]:
        s["table"] = torch.randperm(s["pages"], generator=gen, device="cuda")[:B * pps].view(B, pps).to(torch.int32)
        for key in ("k_codes", "k_sz", "v_codes", "v_sz"):
            if s[key] is not None:
                rows = s[key].unflatten(2, (pps, PAGE)).transpose(1, 2)
                pool = torch.zeros(s["pages"], *rows.shape[2:], dtype=rows.dtype, device="cuda")
                pool[s["table"].long()] = rows
                s[key] = pool
    return s


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "table":
        # what distinguishes two models of a kind: where their context ended and how far it is stretched
        rng = random.Random(int(seed))
        s = {"orig": float(rng.randint(2048, 8192)), "low": 1.0, "high": 4.0 if c["kind"] == "smooth" else 32.0,
             "attn": 1.0 + 0.2 * rng.random(), "table": torch.zeros(c["rows"], c["rot"] // 2, 2, device="cuda")}
    else:
        s = {"plan": _prepare_plan, "append": _prepare_append, "attend": _prepare_attend}[c["op"]](c, gen, int(seed))
    return {"case": c, **s}


# ------------------------------------------------------------------ the plain forms
def _plan_plain(s):
    c = s["case"]
    B, pps, cap = c["B"], c["pps"], s["cap"]
    lens, new, table, dev = s["lens"].long(), s["new"].long(), s["table"], s["lens"].device
    ok = (lens >= 0) & (new >= 0) & (lens + new <= pps * PAGE)
    new = torch.where(ok, new, 0)
    old = (lens.clamp(min=0) + PAGE - 1) // PAGE
    need = torch.where(ok, (lens + new + PAGE - 1) // PAGE - old, 0)
    count = s["free_count"].long().clamp(0, s["free"].numel())
    fits = (new.cumsum(0) <= cap) & (need.cumsum(0) <= count)
    new, need = torch.where(fits, new, 0), torch.where(fits, need, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), new.cumsum(0)])
    page0 = need.cumsum(0) - need
    at = torch.arange(pps, device=dev)
    which = count - 1 - (page0[:, None] + at - old[:, None])
    fresh = (at >= old[:, None]) & (at < (old + need)[:, None])
    table.copy_(torch.where(fresh, s["free"][which.clamp(0, s["free"].numel() - 1)], table))
    t = torch.arange(cap, device=dev)
    here = t < cu[-1]
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=B - 1)
    pos = lens[b] + t - cu[b]
    page = table[b, (pos // PAGE).clamp(0, pps - 1)].long()
    slot = torch.where((page >= 0) & (page < s["pages"]), page * PAGE + pos % PAGE, -1)
    s["new_lens"].copy_(s["lens"] + new)
    s["cu"].copy_(cu)
    s["pos"].copy_(torch.where(here, pos, s["pos"]))
    s["seq"].copy_(torch.where(here, b, s["seq"]))
    s["slots"].copy_(torch.where(here, slot, s["slots"]))
    s["left"].copy_(count - need.sum())
    s["status"].copy_(torch.where((ok & fits).all(), 0, 1))
    return {k: s[k] for k in ("table", "new_lens", "cu", "pos", "seq", "slots", "left", "status")}


def _table_plain(s):
    c = s["case"]
    half, factor, dev = c["rot"] // 2, c["factor"], s["table"].device
    i = torch.arange(half, device=dev, dtype=torch.float64)
    f = c["base"] ** (-i / half)
    if c["kind"] == "linear":
        f = f / factor
    elif c["kind"] == "smooth":
        mix = ((s["orig"] * f / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        f = (1 - mix) * f / factor + mix * f
    elif c["kind"] == "ramp":
        turn = lambda n: c["rot"] * math.log(s["orig"] / (n * 2 * math.pi)) / (2 * math.log(c["base"]))  # noqa: E731
        lo, hi = max(math.floor(turn(s["high"])), 0), min(math.ceil(turn(s["low"])), c["rot"] - 1)
        mix = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * mix + f * (1 - mix)
    # far positions need 64 bits: an angle of 1e5 has only 7 bits of fraction left in 32
    angle = torch.arange(c["rows"], device=dev, dtype=torch.float64)[:, None] * f
    s["table"].copy_(torch.stack([angle.cos(), angle.sin()], -1) * s["attn"])
    return s["table"]


def _halved(x):
    return x[..., 0::2] + x[..., 1::2]  # one level of the pairwise sum of adjacent values


def _normed(x, w, eps):
    D = x.shape[-1]
    t = _halved(_halved(_halved(_halved(_halved(_halved(x * x))))))
    t = _halved(t) if D == 128 else t
    return x * (1.0 / torch.sqrt(t * (1.0 / D) + eps)) * w


def _rotated(x, rot, inter, cos, sin):
    if rot == 0:
        return x
    head, rest = x[..., :rot], x[..., rot:]
    a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., :rot // 2], head[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([turned, rest], -1)


def _append_plain(s):
    c = s["case"]
    N, Hkv, dev = s["pos"].numel(), c["Hkv"], s["x"].device
    here = torch.arange(N, device=dev) < s["count"]
    cs = s["table"][s["pos"].long()][:, None]
    turn = lambda x: _rotated(x, c["rot"], c["inter"], cs[..., 0], cs[..., 1]).to(torch.bfloat16)  # noqa: E731
    q, k = s["q"].float(), s["k"].float()
    if c["norm"]:
        q, k = _normed(q, s["weights"][0].float(), s["eps"]), _normed(k, s["weights"][1].float(), s["eps"])
    s["q_out"].copy_(torch.where(here[:, None, None], turn(q), s["q_out"]))
    # tokens without a slot write what is there already into the last page, which no slot names
    stay = here & (s["slots"] >= 0)
    slot = torch.where(stay, s["slots"], (s["pages"] - 1) * s["page_tokens"])
    at = ((slot // s["page_tokens"])[:, None], torch.arange(Hkv, device=dev)[None], (slot % s["page_tokens"])[:, None])
    for name, x, bits in (("k", turn(k), c["kb"]), ("v", s["v"], c["vb"])):
        for buf, row in zip((s[name + "_codes"], s[name + "_sz"]), _rows(x, bits, c["G"])):
            if row is not None:
                keep = stay.view(-1, *[1] * (row.dim() - 1))
                buf[at] = torch.where(keep, row, buf[at])
    return {k: s[k] for k in ("q_out", "k_codes", "k_sz", "v_codes", "v_sz")}


def _logical(s, key):
    """A cache tensor as [B][Hkv][T][...]."""
    x = s[key]
    if x is None or s["table"] is None:
        return x
    return x[s["table"].long()].transpose(1, 2).flatten(2, 3)


def _attend_plain(s):
    c = s["case"]
    B, Hq, Hkv, D, T, N, mq = c["B"], c["Hq"], c["Hkv"], c["D"], s["T"], s["N"], s["max_q"]
    r, dev, cu = Hq // Hkv, s["q"].device, s["cu"].long()
    n, lens, i = cu.diff(), s["lens"].long(), torch.arange(mq, device=s["q"].device)
    q = s["q"][(cu[:-1, None] + i).clamp(max=N - 1)].float()                               # [B, mq, Hq, D]
    q = q.view(B, mq, Hkv, r, D).transpose(1, 2).reshape(B, Hkv, mq * r, D)
    kh = _values(_logical(s, "k_codes"), _logical(s, "k_sz"), c["kb"], D)
    x = ((q @ kh.transpose(-1, -2)) * s["scale"]).view(B, Hkv, mq, r, T)
    del kh
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    t, p = torch.arange(T, device=dev), (lens - n)[:, None] + i                             # p: [B, mq]
    if c["bias"]:
        x = x + s["slopes"].view(Hkv, 1, r, 1) * (t - p[..., None]).float()[:, None, :, None]
    low = torch.zeros_like(p) if s["start"] is None else s["start"].long()[:, None].expand_as(p)
    if c["window"]:
        low = torch.maximum(low, p - c["window"] + 1)
    see = (t <= p[..., None]) & (t >= low[..., None])
    if s["prefix"] is not None:
        see = see | (t < s["prefix"][:, None, None])
    see = see & (t < lens[:, None, None])
    x = torch.where(see[:, None, :, None], x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    vh = _values(_logical(s, "v_codes"), _logical(s, "v_sz"), c["vb"], D)
    o = e.view(B, Hkv, mq * r, T) @ vh
    o = o.view(B, Hkv, mq, r, D) / torch.where(l == 0, 1.0, l)
    lse = (m + torch.log(l)).squeeze(-1)
    # back to one row for each new token
    tok = torch.arange(N, device=dev)
    b = (torch.searchsorted(cu, tok, right=True) - 1).clamp(max=B - 1)
    at = (tok - cu[b]).clamp(max=mq - 1)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4)[b, at].reshape(N, Hq, D))
    s["lse"].copy_(lse.permute(0, 2, 1, 3)[b, at].reshape(N, Hq))
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ the library's calls
def _plan_own(s, lkv, kept):
    c = s["case"]
    lkv.lkv_page_plan(c["B"], c["pps"], s["pages"], s["cap"], s["lens"], s["new"], s["free"], s["free"].numel(), s["free_count"],
                      s["table"], s["new_lens"], s["cu"], s["pos"], s["seq"], s["slots"], s["left"], s["status"])
    return {k: s[k] for k in ("table", "new_lens", "cu", "pos", "seq", "slots", "left", "status")}


def _table_own(s, lkv, kept):
    c = s["case"]
    if not kept:
        kept.append(lkv.lkv_rope_spec(c["kind"], c["rot"], c["base"], c["factor"], s["low"], s["high"], s["orig"], s["attn"]))
    lkv.lkv_rope_table(kept[0], c["rows"], s["table"])
    return s["table"]


def _append_own(s, lkv, kept):
    c = s["case"]
    wq, wk = (s["weights"][0], s["weights"][1]) if c["norm"] else (None, None)
    lkv.lkv_rope_append_kv((c["kb"], c["vb"], c["G"]), s["pos"].numel(), c["Hq"], c["Hkv"], s["pages"], s["page_tokens"], c["D"],
                           s["count"], s["pos"], s["slots"], s["q"], s["k"], s["v"], wq, wk, s["eps"], c["rot"], c["inter"],
                           s["table"], s["table"].shape[0], s["q_out"], s["k_codes"], s["k_sz"], s["v_codes"], s["v_sz"],
                           reciprocal=True)  # what a tensor program's divisions by constants compute
    return {k: s[k] for k in ("q_out", "k_codes", "k_sz", "v_codes", "v_sz")}


def _attend_own(s, lkv, kept):
    c = s["case"]
    spec = (c["kb"], c["vb"], c["G"])
    if not kept:  # the rule and the workspace that a serving program keeps
        size = lkv.lkv_multi_workspace_bytes(spec, c["B"], c["Hq"], c["Hkv"], s["T"], c["D"], s["max_q"])
        kept += [lkv.lkv_score_rule(s["scale"], c["cap"], c["window"], s["slopes"], s["prefix"], s["start"]),
                 torch.zeros(size, dtype=torch.uint8, device="cuda")]
    rule, ws = kept
    if c["paged"]:
        lkv.lkv_decode_attention_multi_paged(spec, c["B"], c["Hq"], c["Hkv"], s["pps"], s["pages"], c["D"], s["max_q"], s["N"],
                                             s["lens"], s["cu"], s["q"], s["table"], s["k_codes"], s["k_sz"], s["v_codes"],
                                             s["v_sz"], rule, s["out"], s["lse"], ws, ws.numel())
    else:
        lkv.lkv_decode_attention_multi(spec, c["B"], c["Hq"], c["Hkv"], s["T"], c["D"], s["max_q"], s["N"], s["lens"], s["cu"],
                                       s["q"], s["k_codes"], s["k_sz"], s["v_codes"], s["v_sz"], rule, s["out"], s["lse"],
                                       ws, ws.numel())
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        from quantized_kv_cache_lkv_b200 import lkv
        call = {"plan": _plan_own, "table": _table_own, "append": _append_own, "attend": _attend_own}[op]
        return call(state, lkv, state.setdefault("kept", []))
    return {"plan": _plan_plain, "table": _table_plain, "append": _append_plain, "attend": _attend_plain}[op](state)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _bits_of(codes, bits, D):
    """Codes of packed rows, read bit by bit."""
    flags = (codes[..., None] >> torch.arange(8, device=codes.device, dtype=torch.uint8)) & 1
    flags = flags.flatten(-2).unflatten(-1, (D, bits)).double()
    return flags @ (2.0 ** torch.arange(bits, device=codes.device, dtype=torch.float64))


def _exact_attend(c, s):
    D, G, r = c["D"], c["G"], c["Hq"] // c["Hkv"]
    out, lse = torch.zeros(s["N"], c["Hq"], D, dtype=torch.float64, device="cuda"), torch.zeros(s["N"], c["Hq"], dtype=torch.float64, device="cuda")
    lens, n, prefix, start = _attend_lens(c)
    first = 0
    for b in range(c["B"]):
        T, q = lens[b], s["q"][first:first + n[b]].double()
        t = torch.arange(T, device="cuda")
        p = T - n[b] + torch.arange(n[b], device="cuda")[:, None]
        see = (t <= p) & (t >= start[b])
        if c["window"]:
            see &= p - t < c["window"]
        see |= t < prefix[b]
        for g in range(c["Hkv"]):
            rows = []
            for key, bits in (("k", c["kb"]), ("v", c["vb"])):
                if s["table"] is None:
                    codes, sz = s[key + "_codes"][b, g, :T], None if bits == 16 else s[key + "_sz"][b, g, :T]
                else:
                    at = s["table"][b].long()
                    codes = s[key + "_codes"][at, g].flatten(0, 1)[:T]
                    sz = None if bits == 16 else s[key + "_sz"][at, g].flatten(0, 1)[:T]
                if bits == 16:
                    rows.append(codes.contiguous().view(torch.bfloat16).double())
                else:
                    sz = sz.double().repeat_interleave(G, 1)
                    rows.append(_bits_of(codes, bits, D) * sz[..., 0] + sz[..., 1])
            for h in range(g * r, g * r + r):
                x = q[:, h] @ rows[0].T * s["scale"]
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["bias"]:
                    x = x - s["slopes"][h].double() * (p - t)
                x = x.masked_fill(~see, float("-inf"))
                lse[first:first + n[b], h] = torch.logsumexp(x, -1)
                out[first:first + n[b], h] = torch.softmax(x, -1).nan_to_num(0.0) @ rows[1]
        first += n[b]
    return {"out": out, "lse": lse}


def _exact_table(c, s):
    half, a = c["rot"] // 2, np.arange(c["rows"], dtype=np.float64)
    got = np.zeros((c["rows"], half, 2))
    for i in range(half):
        f = math.exp(-math.log(c["base"]) * 2 * i / c["rot"])
        if c["kind"] == "linear":
            f /= c["factor"]
        elif c["kind"] == "smooth":
            turns = s["orig"] / (2 * math.pi / f)
            mix = min(1.0, max(0.0, (turns - s["low"]) / (s["high"] - s["low"])))
            f = f / c["factor"] + mix * (f - f / c["factor"])
        elif c["kind"] == "ramp":
            dim = [c["rot"] / 2 * math.log(s["orig"] / (2 * math.pi * n), c["base"]) for n in (s["high"], s["low"])]
            lo, hi = max(math.floor(dim[0]), 0), min(math.ceil(dim[1]), c["rot"] - 1)
            mix = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f + mix * (f / c["factor"] - f)
        got[:, i, 0], got[:, i, 1] = s["attn"] * np.cos(a * f), s["attn"] * np.sin(a * f)
    return got


def _exact_append(c, s):
    q = s["q"][:c["N"]].double()
    if c["norm"]:
        q = q / torch.sqrt((q * q).mean(-1, keepdim=True) + s["eps"]) * s["weights"][0].double()
    rot, half = c["rot"], c["rot"] // 2
    got = q.clone()
    if rot:
        cs = s["table"].double()[s["pos"][:c["N"]].long()]
        z = torch.complex(cs[..., 0], cs[..., 1])[:, None]
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
        w = torch.complex(q[..., a], q[..., b]) * z
        got[..., a], got[..., b] = w.real, w.imag
    rows = torch.zeros(c["cap"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    rows[:c["N"]] = got
    # codes, scales and zeros hang on roundings of the fixed 32-bit formula: they have no value in 64 bits
    return {"q_out": rows, "k_codes": None, "k_sz": None, "v_codes": None, "v_sz": None}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "plan":
        return None  # whole numbers
    return {"table": _exact_table, "append": _exact_append, "attend": _exact_attend}[c["op"]](c, s)
