"""lkv_decode_attention_multi: caps far above and below the scores, and a distance
bias without near tokens."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_gpu_multi import Cache, call, close, close_lse, cu32, make_q
from quantized_kv_cache_lkv_b200 import lkv

pytestmark = pytest.mark.gpu
SCALE = float(np.float32(128 ** -0.5))


@pytest.mark.parametrize("kb,vb", [(6, 4), (16, 16)])
@pytest.mark.parametrize("cap", [60.0, 1e3, 1e6, 1e20, 1e30, 1e31, 1e33, 1e36, 2.4e38, 3.4e38])
def test_caps_above_the_scores(orc, kb, vb, cap):
    """c * tanh(x / c) is x to fp32 from c = 1e4 on; no cap is too large.  Rows of zeros score exactly 0."""
    cache = Cache(orc, kb, vb, 64, (300, 33), 2, 128, 302, 3)
    q = make_q(2, 8, 128, 4)
    q[1, :4] = 0
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(128 ** -0.5, softcap=cap), 1)
    want, wl = ref.attention(q.float().numpy(), cache.khat, cache.vhat, (300, 33), None, SCALE, softcap=float(np.float32(cap)))
    close(out.cpu().numpy(), want, cache.vmax, f"cap {cap}")
    close_lse(lse.cpu().numpy(), wl)


@pytest.mark.parametrize("cap", [1e-30, 1e-10, 0.5])
def test_caps_below_the_scores(orc, cap):
    cache = Cache(orc, 6, 4, 64, (300, 33), 2, 128, 302, 5)
    q = make_q(2, 8, 128, 6)
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(128 ** -0.5, softcap=cap), 1)
    want, wl = ref.attention(q.float().numpy(), cache.khat, cache.vhat, (300, 33), None, SCALE, softcap=float(np.float32(cap)))
    close(out.cpu().numpy(), want, cache.vmax, f"cap {cap}")
    close_lse(lse.cpu().numpy(), wl)


def test_bias_with_nothing_but_a_far_prefix(orc):
    """Scores of -1e5: all that a query sees is a prefix 100000 positions back, under a bias of 1 a position.  A score is
    then rounded twice at 2^17 binary orders, each time by half of 2^-6: 2^-6 x ln 2 = 1.1e-2 of a weight at most, and of
    the sum of the magnitudes twice that (a weight and the sum of the weights)."""
    T, pre = 100040, 40
    cache = Cache(orc, 6, 4, 64, (T,), 1, 128, T, 7)
    q = make_q(1, 2, 128, 8)
    slopes = np.ones(2, np.float32)
    rule = lkv.lkv_score_rule(128 ** -0.5, slopes=torch.from_numpy(slopes).cuda(), prefix_lens=cu32([pre]), doc_starts=cu32([T]))
    out, lse, _ = call(cache, q.cuda(), None, rule, 1)
    kw = dict(slopes=slopes, prefix=(pre,), starts=(T,))
    want, wl = ref.attention(q.float().numpy(), cache.khat, cache.vhat, (T,), None, SCALE, **kw)
    mag, _ = ref.attention(q.float().numpy(), cache.khat, np.abs(cache.vhat), (T,), None, SCALE, **kw)
    assert (np.abs(out.cpu().numpy() - want) <= 2.2e-2 * mag).all()
    close_lse(lse.cpu().numpy(), wl)
