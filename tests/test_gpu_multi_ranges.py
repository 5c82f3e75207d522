"""lkv_decode_attention_multi where the magnitudes of a cache lie far apart: V rows
or channel groups much larger than the others, whatever weight they get.

Every channel is held against the sum of the magnitudes that enter it,
sum_t w_t |vhat_t|, so that a small row, head or channel group is not hidden
behind a large one.  The bound is the 1e-5 of the other attention tests: the
scores here are at most 8 from their row's largest where they matter, and a
few 2^-24 of the sum of |q khat| (about 10, in units of the binary exponent)
enter exp as 5e-6; exp itself and the two fp16 terms of e * scale add 2^-22
each, the fp32 sums a few 2^-24.

A cached value is itself a sum that may cancel, scale * code + zero.  Its two
terms are each at most |zero| + qmax * scale =: a: the expected value is rounded
twice in fp32 (2^-24 a each), the kernel's product keeps 2^-22 a and its zero of
the middle code 2^-24 a.  All in all 7/16 of 2^-20 a: sum_t w_t a_t 2^-21 is added
to the bound."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_gpu_multi import Cache, call, close_lse
from quantized_kv_cache_lkv_b200 import lkv
from quantized_kv_cache_lkv_b200 import workloads as W

pytestmark = pytest.mark.gpu
REL = 1e-5


def cached(orc, kb, vb, G, k, v, lens):
    """A contiguous cache of K and V [B][Hkv][T][D] rounded to bf16, at any widths, and what it stands for."""
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c = Cache.__new__(Cache)
    D = k.shape[-1]
    p = orc.quantize_kv(kb, vb, G, W.bf16_bits(k), W.bf16_bits(v), np.full(k.shape[0], k.shape[2], np.int32))
    c.kb, c.vb, c.G, c.T_cap, c.lens, c.table, c.host = kb, vb, G, k.shape[2], lens, None, p
    c.khat = k.float().numpy() if kb == 16 else orc.dequant_rows(p["k_codes"], p["k_sz"], D, G, kb)
    c.vhat = v.float().numpy() if vb == 16 else orc.dequant_rows(p["v_codes"], p["v_sz"], D, G, vb)
    c.t = {key: None if (key, 16) in (("k_sz", kb), ("v_sz", vb)) else torch.from_numpy(x).cuda() for key, x in p.items()}
    return c


def weights_and_values(q, cache, lens, cu, scale, **kw):
    """(out, lse, sum_t w_t (|vhat_t| + a_t 2^-21 / REL)) in fp64."""
    out, lse = ref.attention(q, cache.khat, cache.vhat, lens, cu, scale, **kw)
    each = np.abs(cache.vhat).astype(np.float64)
    if cache.vb < 16:
        sz = cache.host["v_sz"].astype(np.float64)
        a = np.abs(sz[..., 1]) + (2 ** cache.vb - 1) * sz[..., 0]
        each += np.repeat(a, cache.G, -1) * 2.0 ** -21 / REL
    mag, _ = ref.attention(q, cache.khat, each, lens, cu, scale, **kw)
    return out, lse, mag


def check(got, lse, q, cache, lens, cu, scale, **kw):
    want, wl, mag = weights_and_values(q.float().numpy(), cache, lens, cu, scale, **kw)
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert np.isfinite(err).all()
    worst = np.unravel_index(np.argmax(err / np.maximum(mag, 1e-300)), err.shape)
    assert (err <= REL * mag).all(), f"{(err / np.maximum(mag, 1e-300)).max():.2e} of the magnitudes at {worst}"
    close_lse(lse.cpu().numpy(), wl)


def make(B, Hkv, T, D, r, n, seed):
    """K and V ~ N(0, 1), and queries that are alike for the heads of a group."""
    gen = torch.Generator().manual_seed(seed)
    k, v = torch.randn(B, Hkv, T, D, generator=gen), torch.randn(B, Hkv, T, D, generator=gen)
    q = torch.randn(B * n, Hkv, 1, D, generator=gen).expand(-1, -1, r, -1).reshape(B * n, Hkv * r, D).to(torch.bfloat16)
    return k, v, q


def against(k, q, at, score, scale, r, n):
    """Puts K rows `at` (of every sequence) where the sequence's first query scores them `score`."""
    qf = q.float().view(k.shape[0], n, k.shape[1], r, -1)[:, 0, :, 0]
    k[:, :, at] = (score / scale * qf / (qf * qf).sum(-1, keepdim=True))[:, :, None]


@pytest.mark.parametrize("kb,vb,G", [(6, 4, 64), (8, 8, 32), (6, 2, 128), (16, 6, 64), (4, 16, 64)])
@pytest.mark.parametrize("power", [0, 8, 16, 30, 60])
@pytest.mark.parametrize("B,T,every", [(1, 32, 1000), (2, 400, 32), (160, 200, 64)])
def test_large_v_without_weight(orc, kb, vb, G, power, B, T, every):
    """Tokens whose V is 2^power times larger and whose weight is e^-100: in the only tile, in every tile, and early in
    runs of several tiles."""
    Hkv, r, D = (4 if B > 2 else 2), 2, 128
    scale = float(np.float32(D ** -0.5))
    k, v, q = make(B, Hkv, T, D, r, 1, power + B)
    big = torch.arange(5, T, every)
    v[:, :, big] *= 2.0 ** power
    against(k, q, big, -100.0, scale, r, 1)
    cache = cached(orc, kb, vb, G, k, v, [T] * B)
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(D ** -0.5), 1)
    check(out, lse, q, cache, [T] * B, None, scale)


@pytest.mark.parametrize("vb", [4, 8])
@pytest.mark.parametrize("n", [2, 4])
def test_large_v_of_another_row(orc, vb, n):
    """A token that only the first query of a sequence still sees: the others' outputs do not feel its size."""
    D, T, scale = 128, 70, float(np.float32(128 ** -0.5))
    k, v, q = make(2, 1, T, D, 4, n, vb + n)
    v[:, :, 0] *= 2.0 ** 24
    cache = cached(orc, 6, vb, 64, k, v, [T, T])
    cu, window = np.arange(3) * n, T - n + 1
    out, lse, _ = call(cache, q.cuda(), cu, lkv.lkv_score_rule(D ** -0.5, window=window), n)
    check(out, lse, q, cache, [T, T], cu, scale, window=window)


@pytest.mark.parametrize("kb,vb,G,D", [(6, 4, 64, 128), (6, 4, 32, 128), (8, 8, 32, 64), (4, 2, 32, 128)])
@pytest.mark.parametrize("power", [-30, -12, 12, 30, 60])
def test_groups_of_different_size(orc, kb, vb, G, D, power):
    """One channel group of every row 2^power times the others: each is exact to its own size."""
    T, scale = 300, float(np.float32(D ** -0.5))
    k, v, q = make(2, 2, T, D, 4, 1, G + D)
    v[..., :G] *= 2.0 ** power
    cache = cached(orc, kb, vb, G, k, v, [T, 33])
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(D ** -0.5), 1)
    check(out, lse, q, cache, [T, 33], None, scale)


@pytest.mark.parametrize("vb", [4, 8])
@pytest.mark.parametrize("how", ["falling", "rising", "early"])
def test_sizes_that_change_along_a_sequence(orc, vb, how):
    """V that shrinks or grows by 2^60 while the scores do the opposite by 60 binary orders, and a first token that
    outweighs everything until a later one outweighs it."""
    D, T, r = 128, 600, 2
    scale = float(np.float32(D ** -0.5))
    k, v, q = make(24, 8, T, D, r, 1, 9)
    at = torch.arange(T)
    ramp = at.float() / T * 60.0
    if how == "early":
        v[:, :, 0] *= 2.0 ** 40
        against(k, q, at[1:2], 30.0, scale, r, 1)
        against(k, q, at[:1], 0.0, scale, r, 1)
    else:
        up = ramp if how == "rising" else 60.0 - ramp
        v = v * torch.exp2(up)[:, None]
        qf = q.float().view(24, 1, 8, r, D)[:, 0, :, 0]
        along = qf / (qf * qf).sum(-1, keepdim=True)
        k = 0.1 * k + (-up * np.log(2.0) / scale)[:, None] * along[:, :, None]
    cache = cached(orc, 16, vb, 64, k, v, [T] * 24)
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(D ** -0.5), 1)
    want, wl, mag = weights_and_values(q.float().numpy(), cache, [T] * 24, None, scale)
    err = np.abs(out.cpu().numpy().astype(np.float64) - want)
    # scores down to -60 binary orders from 16-bit K: exact products in eight sums that each keep 2^-23 of at most 60,
    # 8 x 60 x 2^-23 x ln 2 = 4e-5, beside the 1e-5 of the others
    assert (err <= 5 * REL * mag).all(), f"{(err / np.maximum(mag, 1e-300)).max():.2e}"
    close_lse(lse.cpu().numpy(), wl)


@pytest.mark.parametrize("power", [8, 16])
def test_long_peaky_context(orc, power):
    """131072 tokens with scores of standard deviation 3, one row in 1000 with a large V."""
    D, T = 128, 131072
    k, v, q = make(1, 1, T, D, 2, 1, 4)
    v[:, :, ::1000] *= 2.0 ** power
    cache = cached(orc, 6, 4, 64, k, v, [T])
    scale = float(np.float32(3.0 * D ** -0.5))
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(3.0 * D ** -0.5), 1)
    want, wl, mag = weights_and_values(q.float().numpy(), cache, [T], None, scale)
    err = np.abs(out.cpu().numpy().astype(np.float64) - want)
    # scores of three times the size: three times the bound
    assert (err <= 3 * REL * mag).all(), f"{(err / np.maximum(mag, 1e-300)).max():.2e}"
    close_lse(lse.cpu().numpy(), wl)


@pytest.mark.parametrize("vb", [4, 8])
@pytest.mark.parametrize("jump", [300.0, 1e6, 1e9, 1e20])
def test_scores_that_jump(orc, vb, jump):
    """One token's score passes all before it by far (past what fp32 numbers one by one), in a later tile of the run."""
    D, T, scale = 128, 600, float(np.float32(128 ** -0.5))
    k, v, q = make(24, 8, T, D, 2, 1, 12)
    against(k, q, torch.arange(399, 400), jump, scale, 2, 1)
    cache = cached(orc, 16, vb, 64, k, v, [T] * 24)
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(D ** -0.5), 1)
    want, wl, mag = weights_and_values(q.float().numpy(), cache, [T] * 24, None, scale)
    # the token's weight is 1: e^-300 and less for the others
    assert (np.abs(out.cpu().numpy() - want) <= REL * mag).all()
    # an lse of that size is off by 2^-24 of it for each of the eight sums of its score and for the logarithm's factor
    assert (np.abs(lse.cpu().numpy() - wl) <= 1e-5 * (1 + np.abs(wl))).all()


@pytest.mark.parametrize("vb,G", [(4, 64), (8, 32)])
@pytest.mark.parametrize("power", [-118, -112, -100, -60, 100])
def test_v_near_the_ends_of_fp32(orc, vb, G, power):
    """All of V tiny or huge, while scores of standard deviation 3 rise along the runs."""
    D, T = 128, 600
    k, v, q = make(24, 8, T, D, 2, 1, 13)
    cache = cached(orc, 16, vb, G, k, v * 2.0 ** power, [T] * 24)
    scale = float(np.float32(3.0 * D ** -0.5))
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(3.0 * D ** -0.5), 1)
    want, wl, mag = weights_and_values(q.float().numpy(), cache, [T] * 24, None, scale)
    # scores of three times the size: three times the bound; and the steps of subnormal numbers
    assert (np.abs(out.cpu().numpy() - want) <= 3 * REL * mag + 600 * 2.0 ** -149).all()
    close_lse(lse.cpu().numpy(), wl)
