"""Plain restatements of the serving-step calls for the tests: python loops for
the page plan, numpy fp32 with separate roundings for norm and rotation, numpy
fp64 for the rotary tables and the attention."""
import math

import numpy as np

PAGE = 256


def pages_of(x):
    return -(-x // PAGE)


def page_plan(lens, new, free, count, table, num_pages, n_cap):
    """The outputs of lkv_page_plan as a dict; table is updated in a copy."""
    B, pps = table.shape
    table = table.copy()
    count = min(max(count, 0), len(free))
    out = {"new_lens": lens.copy(), "cu": [0], "pos": [], "seq": [], "slots": []}
    taken, bad, closed = 0, False, False
    for b in range(B):
        L, N = int(lens[b]), int(new[b])
        if L < 0 or N < 0 or L + N > pps * PAGE:
            bad = True
            out["cu"].append(out["cu"][-1])
            continue
        need = pages_of(L + N) - pages_of(L)
        if closed or len(out["pos"]) + N > n_cap or taken + need > count:
            closed = bad = True
            out["cu"].append(out["cu"][-1])
            continue
        for j in range(need):
            table[b, pages_of(L) + j] = free[count - 1 - taken]
            bad |= not 0 <= free[count - 1 - taken] < num_pages
            taken += 1
        for p in range(L, L + N):
            page = int(table[b, p // PAGE])
            ok = 0 <= page < num_pages
            bad |= not ok
            out["pos"].append(p)
            out["seq"].append(b)
            out["slots"].append(page * PAGE + p % PAGE if ok else -1)
        out["new_lens"][b] = L + N
        out["cu"].append(len(out["pos"]))
    return {**out, "table": table, "left": count - taken, "status": int(bad)}


def frequencies(kind, rot, base, factor=1.0, low=1.0, high=32.0, orig=8192.0):
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if kind == "linear":
        return f / factor
    if kind == "smooth":
        w = np.clip((orig * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return (1 - w) * f / factor + w * f
    if kind == "ramp":
        d = lambda n: rot * math.log(orig / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        a, z = max(math.floor(d(high)), 0), min(math.ceil(d(low)), rot - 1)
        w = np.clip((np.arange(rot // 2) - a) / max(z - a, 0.001), 0, 1)
        return w * f / factor + (1 - w) * f
    return f


def bf16(x):
    """fp32 rounded to bf16 (nearest even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def bf16_bits(x):
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def norm_rope(x, weight, eps, rot, inter, cs):
    """x fp32 [N][H][D] -> fp32 holding bf16 values; cs [N][rot / 2][2].  Every operation rounds to fp32."""
    x = x.astype(np.float32)
    D = x.shape[-1]
    if weight is not None:
        t = x * x
        while t.shape[-1] > 1:
            t = t[..., 0::2] + t[..., 1::2]
        r = np.float32(1) / np.sqrt(t * np.float32(1.0 / D) + np.float32(eps))
        x = (x * r) * weight.astype(np.float32)
    x = x.copy()
    if rot:
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        a, b = x[..., ia], x[..., ib]
        c, s = cs[:, None, :, 0], cs[:, None, :, 1]
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return bf16(x)


def quantize_reciprocal(x, bits, G):
    """Codes uint32 [..., D] and (scale, zero) [..., D / G, 2] with products by reciprocals for the divisions."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], -1, G)
    mn, mx = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    d, qmax = mx - mn, np.float32(2 ** bits - 1)
    assert (d > 1e-30).all() and (d < 1e30).all()
    scale, inv = d * (np.float32(1) / qmax), (np.float32(1) / d) * qmax
    codes = np.clip(np.rint((g - mn) * inv), 0, qmax).astype(np.uint32)
    return codes.reshape(x.shape), np.concatenate([scale, mn + np.float32(0)], -1)


def attention(q, khat, vhat, lens, cu, scale, softcap=0.0, window=0, slopes=None, prefix=None, starts=None):
    """fp64 attention of the rows of q [n_rows][Hq][D]; rows outside every sequence give NaN."""
    n_rows, Hq, D = q.shape
    B, Hkv = khat.shape[:2]
    r = Hq // Hkv
    out = np.full((n_rows, Hq, D), np.nan)
    lse = np.full((n_rows, Hq), np.nan)
    for b in range(B):
        c0, c1 = (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))
        T, t = int(lens[b]), np.arange(int(lens[b]))
        for row in range(c0, c1):
            p = T - (c1 - c0) + row - c0
            see = (t <= p) & (t >= (0 if starts is None else int(starts[b])))
            if window:
                see &= p - t < window
            if prefix is not None:
                see |= t < int(prefix[b])
            idx = t[see]
            for h in range(Hq):
                if idx.size == 0:
                    out[row, h], lse[row, h] = 0.0, -np.inf
                    continue
                x = scale * (khat[b, h // r, idx].astype(np.float64) @ q[row, h].astype(np.float64))
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                if slopes is not None:
                    x = x + float(slopes[h]) * (idx - p)
                m = x.max()
                e = np.exp(x - m)
                lse[row, h] = m + np.log(e.sum())
                out[row, h] = (e / e.sum()) @ vhat[b, h // r, idx].astype(np.float64)
    return out, lse
