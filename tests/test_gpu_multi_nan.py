"""lkv_decode_attention_multi where what a query sees is not a number."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_gpu_multi import Cache, call, close, close_lse, make_q
from quantized_kv_cache_lkv_b200 import lkv

pytestmark = pytest.mark.gpu
SCALE = float(np.float32(128 ** -0.5))


@pytest.mark.parametrize("kb,vb,where", [(16, 16, "k"), (16, 4, "k"), (6, 4, "k_sz"), (6, 4, "q"), (16, 16, "q")])
@pytest.mark.parametrize("T", [20, 3000])
def test_nan_that_is_seen_stays_in_sight(orc, kb, vb, where, T):
    """A row whose scores are not numbers has neither an output nor an lse that is one -- -infinity says that a query sees
    nothing -- whether one warp holds it or many; other sequences do not feel it."""
    cache = Cache(orc, kb, vb, 64, (T, 33), 1, 128, T + T % 2 + 34, 9)
    q = make_q(2, 4, 128, 10)
    if where == "q":
        q[0] = float("nan")
    elif where == "k":
        cache.t["k_codes"][0, :, :T] = 0xFF
    else:
        cache.t["k_sz"][0, :, :T, :, 1] = float("nan")
    out, lse, _ = call(cache, q.cuda(), None, lkv.lkv_score_rule(128 ** -0.5), 1)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    want, wl = ref.attention(q.float().numpy()[1:], cache.khat[1:], cache.vhat[1:], (33,), None, SCALE)
    close(out[1:].cpu().numpy(), want, cache.vmax)
    close_lse(lse[1:].cpu().numpy(), wl)
