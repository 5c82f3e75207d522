"""lkv_rope_table against fp64 and lkv_rope_append_kv bit for bit against the
fixed fp32 formula (numpy) and the oracle's quantizer."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from quantized_kv_cache_lkv_b200 import lkv

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ tables
@pytest.mark.parametrize("kind,rot,rows,kw", [
    ("none", 128, 1, {}), ("none", 16, 1000, {}), ("none", 64, 131071, dict(base=500000.0)),
    ("linear", 32, 777, dict(factor=4.0)), ("linear", 128, 255, dict(factor=0.5)),
    ("smooth", 128, 8192, dict(base=500000.0, factor=8.0, low=1.0, high=4.0)),
    ("smooth", 48, 257, dict(factor=2.0, low=1.0, high=4.0, orig_ctx=100.0)),
    ("ramp", 128, 40000, dict(factor=16.0, attn_factor=1.2772588722239782)),
    ("ramp", 96, 513, dict(factor=32.0, orig_ctx=4096.0)), ("ramp", 112, 33, dict(factor=4.0, low=1.0, high=1.5, orig_ctx=10.0)),
])
def test_table_matches_fp64(kind, rot, rows, kw):
    spec = lkv.lkv_rope_spec(kind, rot, **kw)
    table = torch.full((rows + 1, rot // 2, 2), 7.0, device="cuda")
    lkv.lkv_rope_table(spec, rows, table)
    got = table.cpu().numpy()
    assert (got[rows] == 7.0).all(), "a row behind the table was written"
    f = ref.frequencies(kind, rot, spec.base, spec.factor, spec.low, spec.high, spec.orig_ctx)
    angle = np.arange(rows)[:, None] * f
    want = spec.attn_factor * np.stack([np.cos(angle), np.sin(angle)], -1)
    # one rounding to fp32 (2^-24 of the value); the frequency's relative error in
    # fp64, on either side, is below 2 log2(base) 2^-52 (exponent and power) and
    # grows with the angle; 32 + 8 turns of 2^-51 each
    bound = 2.0 ** -24 * np.abs(want) + spec.attn_factor * (4 * np.log2(spec.base) * 2.0 ** -52 * angle.max() + 80 * 2.0 ** -51)
    assert (np.abs(got[:rows] - want) <= bound).all(), np.abs(got[:rows] - want).max()


# ------------------------------------------------------------------ append
def make(N, cap, Hq, Hkv, D, seed, fused=True, outliers=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(cap, Hq + 2 * Hkv, D, generator=gen) * torch.exp(torch.randn(1, Hq + 2 * Hkv, D, generator=gen))
    if outliers:
        x[:, :, 3] *= 40
    x = x.to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(2, D, generator=gen)).to(torch.bfloat16)
    d = x.cuda()
    q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return x, w, q, k, v


def run(orc, kb=6, vb=4, G=64, N=5, cap=None, Hq=8, Hkv=2, D=128, rot=128, inter=False, norm=True, paged=True, seed=0, fused=True,
        slots=None, pos=None, n_tokens="N", table_rows=600, eps=1e-6, reciprocal=False):
    cap = N if cap is None else cap
    x, w, q, k, v = make(N, cap, Hq, Hkv, D, seed, fused)
    rng = np.random.default_rng(seed)
    page_tokens, pages = (256, 3 + N // 128) if paged else (202 + N, 2)
    if slots is None:
        slots = rng.permutation(pages * page_tokens)[:cap]
    if pos is None:
        pos = rng.integers(0, table_rows, cap)
    table = rng.uniform(-1, 1, (table_rows, max(rot // 2, 1), 2)).astype(np.float32)
    ng = D // G
    cache = {"k_codes": torch.full((pages, Hkv, page_tokens, D * kb // 8), 0xA5, dtype=torch.uint8, device="cuda"),
             "k_sz": torch.full((pages, Hkv, page_tokens, ng, 2), 3.5, device="cuda"),
             "v_codes": torch.full((pages, Hkv, page_tokens, D * vb // 8), 0xA5, dtype=torch.uint8, device="cuda"),
             "v_sz": torch.full((pages, Hkv, page_tokens, ng, 2), 3.5, device="cuda")}
    before = {key: t.cpu().numpy() for key, t in cache.items()}
    q_out = torch.full((cap, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    count = None if n_tokens is None else torch.tensor([N if n_tokens == "N" else n_tokens], dtype=torch.int32, device="cuda")
    wd = w.cuda()
    lkv.lkv_rope_append_kv((kb, vb, G), cap, Hq, Hkv, pages, page_tokens, D, count,
                           torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(slots, dtype=torch.int64, device="cuda"),
                           q, k, v, wd[0] if norm else None, wd[1] if norm else None, eps, rot, inter,
                           torch.from_numpy(table).cuda(), table_rows, q_out, cache["k_codes"], cache["k_sz"],
                           cache["v_codes"], cache["v_sz"], reciprocal=reciprocal)
    torch.cuda.synchronize()
    # the formula
    n = cap if count is None else min(max(int(count), 0), cap)
    keep = np.array([t < n and (rot == 0 or 0 <= pos[t] < table_rows) for t in range(cap)], bool)
    xf, wf = x.float().numpy(), w.float().numpy()
    cs = table[np.clip(pos, 0, table_rows - 1)]
    want_q = np.full((cap, Hq, D), 9.0, np.float32)
    want_q[keep] = ref.norm_rope(xf[:, :Hq], wf[0] if norm else None, eps, rot, inter, cs)[keep]
    np.testing.assert_array_equal(ref.bf16_bits(q_out.float().cpu().numpy()), ref.bf16_bits(want_q))
    kr = ref.norm_rope(xf[:, Hq:Hq + Hkv], wf[1] if norm else None, eps, rot, inter, cs)
    bits = lambda y: np.ascontiguousarray(ref.bf16_bits(y).transpose(1, 0, 2)[None])  # noqa: E731  [1][Hkv][cap][D]
    if reciprocal:
        o = {}
        for key, y, b in (("k", kr, kb), ("v", xf[:, Hq + Hkv:], vb)):
            codes, sz = ref.quantize_reciprocal(y.transpose(1, 0, 2)[None], b, G)
            o[key + "_codes"] = np.stack([orc.pack_row(row, b) for row in codes.reshape(-1, D)]).reshape(1, Hkv, cap, -1)
            o[key + "_sz"] = sz
    else:
        o = orc.quantize_kv(kb, vb, G, bits(kr), bits(xf[:, Hq + Hkv:]), np.array([cap], np.int32))
    want = before
    for t in range(cap):
        if keep[t] and 0 <= slots[t] < pages * page_tokens:
            page, off = divmod(int(slots[t]), page_tokens)
            for key in want:
                if not (key == "k_sz" and kb == 16 or key == "v_sz" and vb == 16):
                    want[key][page, :, off] = o[key][0, :, t].reshape(want[key][page, :, off].shape)
    for key in want:
        got = cache[key].cpu().numpy()
        assert np.array_equal(got.view(np.uint8), want[key].view(np.uint8)), key


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 80, 96, 112, 128])
def test_rotations(orc, D, inter, rot):
    if rot > D:
        pytest.skip("more channels than the head has")
    run(orc, D=D, G=64, rot=rot, inter=inter, norm=rot % 32 == 0, seed=rot + D)


@pytest.mark.parametrize("kb", [2, 4, 6, 8, 16])
@pytest.mark.parametrize("vb", [2, 4, 6, 8, 16])
def test_widths(orc, kb, vb):
    G = {2: 32, 4: 64, 6: 128, 8: 64, 16: 32}[kb]
    run(orc, kb=kb, vb=vb, G=G, seed=kb * 20 + vb, N=3, Hkv=3, Hq=3)
    run(orc, kb=kb, vb=vb, G=32, D=64, rot=64, seed=kb * 20 + vb, N=2, Hkv=5, Hq=5, inter=True)


@pytest.mark.parametrize("kb,vb,G", [(6, 4, 64), (8, 2, 32), (4, 8, 128)])
def test_reciprocal_quantizer(orc, kb, vb, G):
    run(orc, kb=kb, vb=vb, G=G, N=200, seed=kb, reciprocal=True)


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (17, 6, 2), (300, 7, 7), (2600, 17, 1)])
def test_batches(orc, N, Hq, Hkv):
    """One token to runs of four row batches a warp, heads that do not fill a warp."""
    run(orc, N=N, Hq=Hq, Hkv=Hkv, D=64 if N > 1000 else 128, rot=32, seed=N)


@pytest.mark.parametrize("paged,fused", [(True, False), (False, True), (False, False)])
def test_layouts(orc, paged, fused):
    run(orc, paged=paged, fused=fused, N=9, seed=5)


@pytest.mark.parametrize("n_tokens", [None, 0, 3, 99, -2])
def test_padded_batch_leaves_the_rest(orc, n_tokens):
    run(orc, N=5, cap=8, n_tokens=n_tokens, seed=7)


def test_slots_and_positions_out_of_range(orc):
    run(orc, N=8, slots=np.array([5, -1, 9, 1 << 40, 700, -(1 << 40), 256, 1023 * 256]), pos=np.array([0, 599, 600, -1, 3, 4, 1 << 30, 5]))


def test_zero_rows_and_large_values(orc):
    """A head of zeros stays zeros through the norm; eps 0 is allowed for the others."""
    x, w, q, k, v = make(4, 4, 4, 2, 128, 3)
    q[1] = 0
    k[2] = 0
    out = torch.empty(4, 4, 128, dtype=torch.bfloat16, device="cuda")
    c = [torch.zeros(1, 2, 256, 96, dtype=torch.uint8, device="cuda"), torch.ones(1, 2, 256, 2, 2, device="cuda"),
         torch.zeros(1, 2, 256, 64, dtype=torch.uint8, device="cuda"), torch.ones(1, 2, 256, 2, 2, device="cuda")]
    lkv.lkv_rope_append_kv((6, 4, 64), 4, 4, 2, 1, 256, 128, None, None, torch.arange(4, device="cuda"), q, k, v, w.cuda()[0],
                           w.cuda()[1], 1e-6, 0, 0, None, 0, out, *c)
    assert (out[1] == 0).all() and (c[1][0, :, 2] == 0).all() and torch.isfinite(out.float()).all()


def test_two_calls_on_two_streams(orc):
    """Two batches into one cache at the same time, from the streams that made them."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    c = [torch.zeros(2, 2, 256, 96, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, 256, 2, 2, device="cuda"),
         torch.zeros(2, 2, 256, 64, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, 256, 2, 2, device="cuda")]
    one = [t.clone() for t in c]
    torch.cuda.synchronize()
    outs = []
    for i, s in enumerate((a, b)):
        with torch.cuda.stream(s):
            x, w, q, k, v = make(256, 256, 4, 2, 128, 40 + i)
            out = torch.empty(256, 4, 128, dtype=torch.bfloat16, device="cuda")
            for dst in (c, one):
                lkv.lkv_rope_append_kv((6, 4, 64), 256, 4, 2, 2, 256, 128, None, None, torch.arange(256, device="cuda") + 256 * i,
                                       q, k, v, w.cuda()[0], w.cuda()[1], 1e-6, 0, 0, None, 0, out, *dst)
            outs.append(out)
    torch.cuda.synchronize()
    for x, y in zip(c, one):
        assert torch.equal(x, y)


@pytest.mark.parametrize("D,rot", [(64, 0), (64, 16), (64, 48), (128, 0), (128, 16), (128, 48), (128, 80), (128, 112)])
@pytest.mark.parametrize("N", [3, 1500])
def test_norm_with_some_channels_turning(orc, D, rot, N):
    """The norm's sum runs over adjacent channels while the lanes hold pairs; large calls take runs of heads."""
    run(orc, N=N, Hq=33, Hkv=5, D=D, G=32, rot=rot, norm=True, seed=N + rot)
