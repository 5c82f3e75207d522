"""lkv_decode_attention_multi, contiguous and paged, against numpy fp64 over the
dequantized cache.  Tolerances are the decode's: rel-L2 1e-5 and 5e-5 of the
largest |V| (fp32 arithmetic; the scores' fp32 rounding, a few 2^-24 of scores
up to about 40, enters exp as 1e-5 at most)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from quantized_kv_cache_lkv_b200 import buffers, lkv
from quantized_kv_cache_lkv_b200 import workloads as W

pytestmark = pytest.mark.gpu
P = lkv.LKV_PAGE_TOKENS
REL, ABS = 1e-5, 5e-5


def cu32(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Cache:
    """A packed cache made by the oracle's quantizer, contiguous or in shuffled pages, and what it stands for."""

    def __init__(self, orc, kb, vb, G, lens, Hkv, D, T_cap, seed, paged=False, poison=False):
        B = len(lens)
        cfg = W.Config("multi", B=B, Hq=Hkv, Hkv=Hkv, D=D, T_cap=T_cap, G=G, bits=[(kb, vb)], hh_frac=0.01, seed=seed)
        inp = W.make_inputs(cfg, seq_lens=torch.tensor(lens, dtype=torch.int32))
        k, v = W.bf16_bits(inp["k"]), W.bf16_bits(inp["v"])
        c = orc.quantize_kv(kb, vb, G, k, v, np.full(B, T_cap, np.int32))
        self.kb, self.vb, self.G, self.T_cap, self.lens, self.pps = kb, vb, G, T_cap, lens, T_cap // P
        self.khat = orc.dequant_rows(c["k_codes"], c["k_sz"], D, G, kb) if kb < 16 else inp["k"].float().numpy()
        self.vhat = orc.dequant_rows(c["v_codes"], c["v_sz"], D, G, vb) if vb < 16 else inp["v"].float().numpy()
        self.vmax = float(np.abs(self.vhat).max()) or 1.0
        if poison:  # nothing that no query sees may matter
            for b, T in enumerate(lens):
                self.hide(c, b, slice(T, None))
        t = {}
        for key, rows, bits in (("k_codes", D * kb // 8, kb), ("k_sz", 0, kb), ("v_codes", D * vb // 8, vb), ("v_sz", 0, vb)):
            if key.endswith("sz") and bits == 16:
                t[key] = None
            else:
                t[key] = torch.from_numpy(np.ascontiguousarray(c[key]).reshape(B, Hkv, T_cap, -1 if rows else D // G, *([] if rows else [2])))
        self.table, self.num_pages = None, 0
        if paged:
            self.num_pages = B * self.pps + 2
            table = torch.randperm(self.num_pages, generator=torch.Generator().manual_seed(seed))[:B * self.pps].view(B, self.pps)
            for key, x in t.items():
                if x is not None:
                    pool = torch.zeros(self.num_pages, Hkv, P, *x.shape[3:], dtype=x.dtype)
                    if poison and x.dtype == torch.float32:
                        pool.fill_(float("nan"))
                    pool[table] = x.unflatten(2, (self.pps, P)).transpose(1, 2)
                    t[key] = pool
            self.table = table.to(torch.int32).cuda()
        self.t = {key: None if x is None else x.cuda() for key, x in t.items()}
        self.host = c

    def hide(self, c, b, rows):
        for key, bits in (("k", self.kb), ("v", self.vb)):
            if bits == 16:
                c[key + "_codes"][b, :, rows] = 0xFF  # bf16 NaN
            else:
                c[key + "_sz"][b, :, rows] = np.where(np.arange(2) == 0, np.nan, np.inf)


def call(cache, q, cu, rule, max_q, ws=None, lse=True, seq_lens=None, stream=None, fill=5.0):
    n_rows, Hq, D = q.shape
    Hkv = cache.khat.shape[1]
    B = len(cache.lens)
    spec = (cache.kb, cache.vb, cache.G)
    out = torch.full((n_rows, Hq, D), fill, device="cuda")
    ls = torch.full((n_rows, Hq), fill, device="cuda") if lse else None
    if ws is None:
        ws = buffers.alloc_workspace(lkv.lkv_multi_workspace_bytes(spec, B, Hq, Hkv, cache.T_cap, D, max_q))
    t, sl = cache.t, cu32(cache.lens if seq_lens is None else seq_lens)
    rest = (t["k_codes"], t["k_sz"], t["v_codes"], t["v_sz"], rule, out, ls, ws, ws.numel())
    if cache.table is None:
        lkv.lkv_decode_attention_multi(spec, B, Hq, Hkv, cache.T_cap, D, max_q, n_rows, sl, cu32(cu), q, *rest, stream=stream)
    else:
        lkv.lkv_decode_attention_multi_paged(spec, B, Hq, Hkv, cache.pps, cache.num_pages, D, max_q, n_rows, sl, cu32(cu), q,
                                             cache.table, *rest, stream=stream)
    torch.cuda.synchronize()
    return out, ls, ws


def make_q(n_rows, Hq, D, seed):
    return torch.randn(n_rows, Hq, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def close(got, want, vmax, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want)
    live = ~np.isnan(want)
    assert (got[~live] == 5.0).all(), what + ": a row outside every sequence was written"
    got, want = got[live], want[live]
    assert np.isfinite(got).all(), what
    if got.size:
        d, n = np.linalg.norm(got - want), np.linalg.norm(want)
        assert d <= REL * n, f"{what}: rel-L2 {d / max(n, 1e-300):.3e}"
        assert np.abs(got - want).max() <= ABS * vmax, f"{what}: max-abs {np.abs(got - want).max():.3e}"


def close_lse(got, want):
    """ln of a sum of exp: off by the scores' fp32 rounding, at most 1e-5 of 1 + |lse|."""
    got, want = np.asarray(got, np.float64), np.asarray(want)
    live = ~np.isnan(want)
    assert (got[~live] == 5.0).all()
    empty = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), empty)
    live &= ~empty
    assert (np.abs(got[live] - want[live]) <= 1e-5 * (1 + np.abs(want[live]))).all()


def case(orc, kb=6, vb=4, G=64, lens=(300, 1, 77), Hkv=2, r=4, D=128, n=1, paged=False, seed=0, softcap=0.0, slopes=False, window=0,
         prefix=None, starts=None, poison=False, T_cap=None, extra=0, hidden=()):
    B, Hq = len(lens), Hkv * r
    T_cap = T_cap or (-(-max(max(lens), 1) // P) * P if paged else max(lens) + max(lens) % 2 + 2)
    cache = Cache(orc, kb, vb, G, lens, Hkv, D, T_cap, seed, paged, poison)
    ns = [n] * B if isinstance(n, int) else list(n)
    cu = None if n == 1 and not extra else np.cumsum([0] + ns)
    rows = sum(ns) + extra
    q = make_q(rows, Hq, D, seed + 1)
    sl = 2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq) if slopes else None
    rule = lkv.lkv_score_rule(D ** -0.5, softcap, window, None if sl is None else torch.tensor(sl, dtype=torch.float32, device="cuda"),
                              cu32(prefix), cu32(starts))
    out, lse, ws = call(cache, q.cuda(), cu, rule, max(max(ns), 1))
    assert lkv.lkv_workspace_status(ws) == lkv.LKV_OK
    scale = float(np.float32(D ** -0.5))
    want, wl = ref.attention(q.float().numpy(), cache.khat, cache.vhat, lens, cu, scale, softcap, window,
                             None if sl is None else sl.astype(np.float32), prefix, starts)
    close(out.cpu().numpy(), want, cache.vmax, "out")
    close_lse(lse.cpu().numpy(), wl)
    return cache, q, cu, rule, out, lse, ws


@pytest.mark.parametrize("kb", [2, 4, 6, 8, 16])
@pytest.mark.parametrize("vb", [2, 4, 6, 8, 16])
@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
def test_widths_groups_dims(orc, kb, vb, D, G):
    case(orc, kb, vb, G, lens=(70, 1, 33, 16), D=D, Hkv=1, r=2, seed=kb + vb, poison=True)


@pytest.mark.parametrize("r", [1, 2, 3, 4, 5, 7, 8, 16, 64])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_groups_and_runs(orc, r, n):
    case(orc, r=r, n=n, lens=(130, 31, 64) if r < 16 else (65, 9), seed=r + n)


@pytest.mark.parametrize("lens", [(0,), (1,), (2,), (15, 16, 17), (31, 32, 33), (255, 256, 257), (0, 5, 0, 0, 900, 1, 0)])
@pytest.mark.parametrize("paged", [False, True])
def test_lengths(orc, lens, paged):
    case(orc, lens=lens, paged=paged, seed=3, poison=True)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kb,vb,G,D", [(6, 4, 64, 128), (8, 8, 32, 128), (16, 16, 64, 128), (4, 2, 32, 64)])
def test_long_and_ragged(orc, kb, vb, G, D, paged):
    case(orc, kb, vb, G, D=D, lens=(3000, 17, 1025, 512, 2047), paged=paged, seed=11, r=2)


@pytest.mark.parametrize("kw", [
    dict(softcap=30.0), dict(softcap=2.0), dict(softcap=50.0, slopes=True), dict(slopes=True), dict(window=1), dict(window=16),
    dict(window=33, n=4), dict(window=100000), dict(window=20, prefix=(5, 0, 40)), dict(prefix=(300, 77, 1), window=1),
    dict(starts=(100, 0, 76)), dict(starts=(299, 1, 77), n=3), dict(starts=(400, 300, 80)),
    dict(starts=(400, 300, 80), prefix=(0, 3, 1000)), dict(starts=(64, 10, 32), prefix=(32, 16, 3), window=50, n=5, slopes=True, softcap=20.0),
    dict(prefix=(-5, 1 << 30, 77), starts=(-9, 5, 50)),
])
@pytest.mark.parametrize("kb,vb", [(6, 4), (16, 16)])
def test_masks_and_scores(orc, kw, kb, vb):
    kw = dict(kw)
    case(orc, kb, vb, lens=(300, 20, 77), seed=21, poison=True, **kw)


def test_prefix_sees_ahead(orc):
    """Query rows inside the prefix see all of it, later positions too."""
    case(orc, lens=(40, 64), n=20, prefix=(40, 50), seed=31)


def test_more_rows_than_tokens(orc):
    """Rows at negative positions see nothing but the prefix."""
    case(orc, lens=(3, 0, 2), n=5, seed=32)
    case(orc, lens=(3, 0, 2), n=5, prefix=(2, 2, 0), seed=33)


@pytest.mark.parametrize("ns", [(3, 0, 1, 8), (0, 0, 0, 1), (1, 64, 2, 0)])
def test_ragged_rows_and_rows_behind(orc, ns):
    case(orc, lens=(200, 30, 64, 90), n=ns, extra=3, seed=41)


@pytest.mark.parametrize("kb,vb", [(6, 4), (16, 16), (6, 16)])
def test_hidden_rows_may_be_anything(orc, kb, vb):
    """Positions before the document start hold NaN and infinities inside tiles that are read."""
    lens, starts = (100, 50), (37, 20)
    cache = Cache(orc, kb, vb, 64, lens, 2, 128, 102, 5)
    for b in range(2):
        cache.hide(cache.host, b, slice(0, starts[b]))
    for key in cache.t:
        if cache.t[key] is not None:
            cache.t[key].copy_(torch.from_numpy(np.ascontiguousarray(cache.host[key]).reshape(cache.t[key].shape)))
    q = make_q(2, 8, 128, 6)
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(128 ** -0.5, doc_starts=cu32(starts)), 1)
    want, wl = ref.attention(q.float().numpy(), cache.khat, cache.vhat, lens, None, float(np.float32(128 ** -0.5)), starts=starts)
    close(out.cpu().numpy(), want, cache.vmax)
    close_lse(lse.cpu().numpy(), wl)


def test_many_short_sequences(orc):
    """More units than warps: whole units inside one warp's run, cut ones joined inside the CTA."""
    rng = np.random.default_rng(2)
    case(orc, lens=tuple(int(x) for x in rng.integers(0, 120, 700)), Hkv=4, r=1, D=64, G=32, seed=51, kb=4, vb=4)


def test_q_of_zeros_and_tiny_and_large(orc):
    cache = Cache(orc, 6, 4, 64, (90,), 1, 128, 92, 8)
    for scale in (0.0, 2.0 ** -120, 2.0 ** 60):
        q = (make_q(1, 4, 128, 9).float() * scale).to(torch.bfloat16)
        rule = lkv.lkv_score_rule(2.0 ** -60 if scale > 1 else 1.0)
        out, _, _ = call(cache, q.cuda(), None, rule, 1)
        want, _ = ref.attention(q.float().numpy(), cache.khat, cache.vhat, (90,), None, rule.softmax_scale)
        close(out.cpu().numpy(), want, cache.vmax, f"scale {scale}")


def from_values(orc, kb, vb, G, k, v, lens):
    """A contiguous cache of given bf16 K and V [B][Hkv][T][D]."""
    c = Cache.__new__(Cache)
    D = k.shape[-1]
    p = orc.quantize_kv(kb, vb, G, W.bf16_bits(k), W.bf16_bits(v), np.full(k.shape[0], k.shape[2], np.int32))
    c.kb, c.vb, c.G, c.T_cap, c.lens, c.table, c.host = kb, vb, G, k.shape[2], lens, None, p
    c.khat = orc.dequant_rows(p["k_codes"], p["k_sz"], D, G, kb)
    c.vhat = orc.dequant_rows(p["v_codes"], p["v_sz"], D, G, vb)
    c.vmax = float(np.abs(c.vhat).max())
    c.t = {key: torch.from_numpy(x).cuda() for key, x in p.items()}
    return c


@pytest.mark.parametrize("kb,vb,G", [(6, 4, 64), (8, 8, 32), (4, 2, 128), (2, 6, 64)])
@pytest.mark.parametrize("how", ["constant", "rising", "tiny", "huge", "offset"])
def test_ranges_of_v_and_k(orc, kb, vb, G, how):
    """Groups without a range, V whose scales rise by 2^40 along the sequence, V near the ends of fp32, and values far
    from 0 next to their range."""
    gen = torch.Generator().manual_seed(5)
    B, Hkv, T, D = 2, 1, 400, 128
    k, v = torch.randn(B, Hkv, T, D, generator=gen), torch.randn(B, Hkv, T, D, generator=gen)
    if how == "constant":
        k, v = k[..., :1].expand_as(k).clone(), v[..., :1].expand_as(v).clone()
    if how == "rising":
        v = v * torch.exp2(torch.arange(T) * 0.1)[:, None]
    if how == "tiny":
        v = v * 2.0 ** -100
    if how == "huge":
        v = v * 2.0 ** 100
    if how == "offset":
        k, v = k + 5.0, v * 0.01 + 30.0
    cache = from_values(orc, kb, vb, G, k.to(torch.bfloat16), v.to(torch.bfloat16), (T, 33))
    q = make_q(2, 8, D, 6)
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(D ** -0.5), 1)
    want, wl = ref.attention(q.float().numpy(), cache.khat, cache.vhat, (T, 33), None, float(np.float32(D ** -0.5)))
    close(out.cpu().numpy(), want, cache.vmax, how)
    close_lse(lse.cpu().numpy(), wl)


def test_no_capacity():
    """T_cap 0: nothing to see, zeros."""
    out, lse = torch.full((2, 8, 128), 5.0, device="cuda"), torch.full((2, 8), 5.0, device="cuda")
    ws = buffers.alloc_workspace(lkv.lkv_multi_workspace_bytes((6, 4, 64), 2, 8, 2, 0, 128, 1))
    lkv.lkv_decode_attention_multi((6, 4, 64), 2, 8, 2, 0, 128, 1, 2, cu32([0, 0]), None, make_q(2, 8, 128, 1).cuda(), None, None, None, None,
                                   lkv.lkv_score_rule(0.1), out, lse, ws, ws.numel())
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_largest_batch(orc):
    """4096 sequences, most of them short."""
    rng = np.random.default_rng(8)
    case(orc, 4, 4, 64, lens=tuple(int(x) for x in rng.integers(0, 20, 4096)), Hkv=1, r=1, D=64, seed=52)


def test_two_calls_at_once_with_their_own_workspaces(orc):
    """Two streams, two workspaces: each call's result is what it is alone."""
    one = case(orc, lens=(4000, 900), n=2, seed=71)
    two = case(orc, 8, 4, 64, lens=(2500, 1, 3000), r=8, seed=72)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got, keep = [], []
    for _ in range(3):
        for stream, (cache, q, cu, rule, out, lse, ws) in ((s, one), (t, two)):
            rows, Hq, D = q.shape
            o = torch.full_like(out, 5.0)
            c, max_q = cache.t, 2 if cache is one[0] else 1
            lens, offsets, qd = cu32(cache.lens), cu32(cu), q.cuda()
            keep += [lens, offsets, qd]  # until both streams are done with them
            stream.wait_stream(torch.cuda.current_stream())
            lkv.lkv_decode_attention_multi((cache.kb, cache.vb, cache.G), len(cache.lens), Hq, 2, cache.T_cap, D, max_q, rows,
                                           lens, offsets, qd, c["k_codes"], c["k_sz"], c["v_codes"], c["v_sz"], rule, o,
                                           None, ws, ws.numel(), stream=stream)
            got.append((o, out))
    torch.cuda.synchronize()
    for o, want in got:
        assert torch.equal(o, want)


def test_same_result_every_time_and_on_a_used_workspace(orc):
    """Bit-identical on a workspace that calls of other sizes have used, on another stream, and without lse."""
    cache, q, cu, rule, out, lse, _ = case(orc, lens=(5000, 40, 3000), n=3, seed=61)
    other, oq, ocu, orule, oout, _, _ = case(orc, 8, 8, 32, lens=(900,) * 9, n=8, seed=62)
    need = max(lkv.lkv_multi_workspace_bytes((6, 4, 64), 3, 8, 2, cache.T_cap, 128, 3),
               lkv.lkv_multi_workspace_bytes((8, 8, 32), 9, 8, 2, other.T_cap, 128, 8))
    ws = buffers.alloc_workspace(need)
    s = torch.cuda.Stream()
    for i in range(3):
        a, la, _ = call(cache, q.cuda(), cu, rule, 3, ws=ws)
        b, _, _ = call(other, oq.cuda(), ocu, orule, 8, ws=ws, lse=False)
        with torch.cuda.stream(s):
            c, lc, _ = call(cache, q.cuda(), cu, rule, 3, ws=ws)
        assert torch.equal(a, out) and torch.equal(la, lse) and torch.equal(b, oout) and torch.equal(c, out) and torch.equal(lc, lse)


def test_captured_graph_reads_new_lengths(orc):
    cache = Cache(orc, 6, 4, 64, (700, 700), 2, 128, 768, 9, paged=True)
    q, lens = make_q(2, 8, 128, 10).cuda(), cu32([700, 700])
    rule = lkv.lkv_score_rule(128 ** -0.5, window=300)
    ws = buffers.alloc_workspace(lkv.lkv_multi_workspace_bytes((6, 4, 64), 2, 8, 2, 768, 128, 1))
    out = torch.zeros(2, 8, 128, device="cuda")
    t = cache.t
    fn = lambda: lkv.lkv_decode_attention_multi_paged((6, 4, 64), 2, 8, 2, 3, cache.num_pages, 128, 1, 2, lens, None, q, cache.table,  # noqa: E731
                                                      t["k_codes"], t["k_sz"], t["v_codes"], t["v_sz"], rule, out, None, ws, ws.numel())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    for L in ((700, 700), (1, 257), (0, 300)):
        lens.copy_(cu32(L))
        g.replay()
        torch.cuda.synchronize()
        want, _ = ref.attention(q.float().cpu().numpy(), cache.khat, cache.vhat, L, None, float(np.float32(128 ** -0.5)), window=300)
        close(out.cpu().numpy(), want, cache.vmax, str(L))


def test_bad_lengths_rows_and_pages_are_reported(orc):
    """Clamped, reported in the status word, finite; the next call after a reset is clean."""
    cache = Cache(orc, 6, 4, 64, (512, 512), 2, 128, 512, 12, paged=True)
    q = make_q(6, 8, 128, 13).cuda()
    rule = lkv.lkv_score_rule(128 ** -0.5)
    for lens, cu, table in (((513, -1), (0, 3, 6), None), ((512, 512), (0, 5, 3), None), ((512, 512), (-2, 3, 9), None),
                            ((512, 512), (0, 1, 6), None), ((512, 512), (0, 3, 6), -1), ((512, 512), (0, 3, 6), 1 << 30)):
        keep = cache.table.clone()
        if table is not None:
            cache.table[1, 1] = table
        out, _, ws = call(cache, q, cu, rule, 3, seq_lens=lens)
        assert torch.isfinite(out).all()
        assert lkv.lkv_workspace_status(ws) == lkv.LKV_ERR_INVALID_ARG, (lens, cu, table)
        cache.table.copy_(keep)
        lkv.lkv_workspace_reset(ws, ws.numel())
        out, _, ws = call(cache, q, (0, 3, 6), rule, 3, ws=ws)
        assert lkv.lkv_workspace_status(ws) == lkv.LKV_OK
        want, _ = ref.attention(q.float().cpu().numpy(), cache.khat, cache.vhat, (512, 512), (0, 3, 6), float(np.float32(128 ** -0.5)))
        close(out.cpu().numpy(), want, cache.vmax)


def test_offsets_past_32_bits(orc):
    """The last rows of a 16-bit cache of 4.3 GB a tensor (byte offsets past 2^32), seen through a window."""
    D, T_cap, T = 128, (1 << 24) + 512, (1 << 24) + 391
    k = torch.empty(1, 1, T_cap, D * 2, dtype=torch.uint8, device="cuda")
    v = torch.empty(1, 1, T_cap, D * 2, dtype=torch.uint8, device="cuda")
    x = torch.randn(2, 100, D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    for buf, rows in ((k, x[0]), (v, x[1])):
        buf[0, 0, T - 160:] = 0xFF  # NaN outside the window
        buf[0, 0, T - 100:T] = rows.cuda().view(torch.uint8)
    q = make_q(1, 2, D, 5)
    out = torch.zeros(1, 2, D, device="cuda")
    ws = buffers.alloc_workspace(lkv.lkv_multi_workspace_bytes((16, 16, 64), 1, 2, 1, T_cap, D, 1))
    rule = lkv.lkv_score_rule(D ** -0.5, window=100, slopes=torch.tensor([0.01, 0.02], device="cuda"))
    lkv.lkv_decode_attention_multi((16, 16, 64), 1, 2, 1, T_cap, D, 1, 1, cu32([T]), None, q.cuda(), k, None, v, None, rule, out, None,
                                   ws, ws.numel())
    xf = x.float().numpy()[:, None, None]
    want, _ = ref.attention(q.float().numpy(), xf[0], xf[1], (100,), None, float(np.float32(D ** -0.5)),
                            slopes=np.float32([0.01, 0.02]))
    close(out.cpu().numpy(), want, float(np.abs(xf[1]).max()))


def test_serving_step(orc):
    """Plan, rotate + append and attend as a loop would: two steps of a ragged batch (prompts of a few tokens, then
    decodes), in one captured graph, against the formulas over bf16 rows kept on the host."""
    B, Hq, Hkv, D, pps, pages, cap = 4, 8, 2, 128, 4, 20, 64
    kb, vb, G = 8, 8, 32
    gen = torch.Generator().manual_seed(77)
    table = torch.full((B, pps), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(pages, generator=gen).to(torch.int32).cuda(), cu32([pages])
    mk = lambda *s, dt=torch.int32: torch.full(s, -1, dtype=dt, device="cuda")  # noqa: E731
    lens, new, lens2, cu, pos, seq, slots = cu32([0] * B), cu32([0] * B), mk(B), mk(B + 1), mk(cap), mk(cap), mk(cap, dt=torch.int64)
    left, status = mk(1), mk(1)
    rot = torch.zeros(2048, 32, 2, device="cuda")
    lkv.lkv_rope_table(lkv.lkv_rope_spec("smooth", 64, 500000.0, 8.0, 1.0, 4.0, 1024.0), 2048, rot)
    x = torch.zeros(cap, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    w = (1 + 0.1 * torch.randn(2, D, generator=gen)).to(torch.bfloat16).cuda()
    qo, out = torch.zeros(cap, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(cap, Hq, D, device="cuda")
    pool = [torch.zeros(pages, Hkv, P, D, dtype=torch.uint8, device="cuda"), torch.zeros(pages, Hkv, P, 4, 2, device="cuda"),
            torch.zeros(pages, Hkv, P, D, dtype=torch.uint8, device="cuda"), torch.zeros(pages, Hkv, P, 4, 2, device="cuda")]
    ws = buffers.alloc_workspace(lkv.lkv_multi_workspace_bytes((kb, vb, G), B, Hq, Hkv, pps * P, D, 16))
    rule = lkv.lkv_score_rule(D ** -0.5, softcap=30.0, window=300)

    def step():
        lkv.lkv_page_plan(B, pps, pages, cap, lens, new, free, pages, count, table, lens2, cu, pos, seq, slots, left, status)
        lkv.lkv_rope_append_kv((kb, vb, G), cap, Hq, Hkv, pages, P, D, cu[B:], pos, slots, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:],
                               w[0], w[1], 1e-6, 64, False, rot, 2048, qo, *pool)
        lkv.lkv_decode_attention_multi_paged((kb, vb, G), B, Hq, Hkv, pps, pages, D, 16, cap, lens2, cu, qo, table, *pool, rule, out,
                                             None, ws, ws.numel())
        lens.copy_(lens2)
        count.copy_(left)

    step()  # no new tokens: nothing happens, and the library is loaded before the capture
    torch.cuda.synchronize()
    assert int(left) == pages and lens.tolist() == [0] * B
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rows = [[[], []] for _ in range(B)]
    table_h, wf = rot.cpu().numpy(), w.float().cpu().numpy()
    for news in ((16, 3, 0, 9), (1, 1, 16, 1), (1, 1, 1, 1)):
        xs = torch.randn(cap, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)
        x.copy_(xs.cuda())
        new.copy_(cu32(news))
        g.replay()
        torch.cuda.synchronize()
        assert int(status) == 0
        n = sum(news)
        xf, p = xs.float().numpy()[:n], pos.cpu().numpy()[:n]
        kr = ref.norm_rope(xf[:, Hq:Hq + Hkv], wf[1], 1e-6, 64, False, table_h[p])
        qr = ref.norm_rope(xf[:, :Hq], wf[0], 1e-6, 64, False, table_h[p])
        at = 0
        for b, m in enumerate(news):
            assert p[at:at + m].tolist() == list(range(len(rows[b][0]), len(rows[b][0]) + m))
            rows[b][0] += list(kr[at:at + m])
            rows[b][1] += list(xf[at:at + m, Hq + Hkv:])
            at += m
        L = [len(rw[0]) for rw in rows]
        T = max(L)
        kv = np.zeros((2, B, Hkv, T, D), np.float32)
        for b in range(B):
            for s in range(2):
                if L[b]:
                    kv[s, b, :, :L[b]] = np.stack(rows[b][s], 1)
        c = orc.quantize_kv(kb, vb, G, ref.bf16_bits(kv[0]), ref.bf16_bits(kv[1]), np.full(B, T, np.int32))
        kh, vh = orc.dequant_rows(c["k_codes"], c["k_sz"], D, G, kb), orc.dequant_rows(c["v_codes"], c["v_sz"], D, G, vb)
        want, _ = ref.attention(qr, kh, vh, L, np.cumsum([0] + list(news)), float(np.float32(D ** -0.5)), softcap=30.0, window=300)
        close(out[:n].cpu().numpy(), want, float(np.abs(vh).max()))
        assert lens.tolist() == L


@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("kw", [dict(), dict(slopes=True), dict(prefix=(50000,), starts=(59990,)), dict(softcap=5.0, window=40000)])
def test_one_unit_across_the_grid(orc, n, kw):
    """Every CTA holds a piece of the only unit; with a distance bias the references of the pieces rise by thousands."""
    case(orc, lens=(60000,), Hkv=1, n=n, seed=61, **kw)


@pytest.mark.parametrize("kb,vb,D,G", [(8, 8, 128, 32), (16, 16, 128, 64), (4, 2, 64, 32)])
def test_few_units_across_the_grid(orc, kb, vb, D, G):
    """Units of several CTAs whose ends lie inside CTAs: one CTA arrives at two units."""
    case(orc, kb, vb, G, D=D, lens=(9001, 8123, 33), Hkv=1, r=8, n=3, seed=62, slopes=True)
