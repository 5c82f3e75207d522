"""lkv_page_plan against a loop over the sequences: every output bit for bit,
what lies behind the last token left alone, and the cases that do not fit."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from quantized_kv_cache_lkv_b200 import lkv

pytestmark = pytest.mark.gpu
P = lkv.LKV_PAGE_TOKENS


def cu32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def plan(lens, new, pps, free, count=None, num_pages=None, n_cap=None, table=None, stream=None):
    """Outputs of the call as numpy arrays, with the sentinels it started from."""
    B = len(lens)
    count = len(free) if count is None else count
    num_pages = 1 << 20 if num_pages is None else num_pages
    n_cap = max(0, int(np.clip(new, 0, None).sum())) + 5 if n_cap is None else n_cap
    if table is None:
        table = (7000 + np.arange(B * pps)).reshape(B, pps)
    d = {"table": cu32(table).view(B, pps), "new_lens": cu32([-7] * B), "cu": cu32([-7] * (B + 1)), "pos": cu32([-7] * n_cap),
         "seq": cu32([-7] * n_cap), "slots": torch.full((n_cap,), -7, dtype=torch.int64, device="cuda"),
         "left": cu32([-7]), "status": cu32([-7])}
    lkv.lkv_page_plan(B, pps, num_pages, n_cap, cu32(lens), cu32(new), cu32(free), len(free), cu32([count]), d["table"],
                      d["new_lens"], d["cu"], d["pos"], d["seq"], d["slots"], d["left"], d["status"], stream=stream)
    torch.cuda.synchronize()
    want = ref.page_plan(np.asarray(lens, np.int64), np.asarray(new, np.int64), list(free), count, np.asarray(table).reshape(B, pps),
                         num_pages, n_cap)
    return {k: v.cpu().numpy() for k, v in d.items()}, want


def check(got, want):
    n = len(want["pos"])
    for key in ("table", "new_lens", "cu"):
        np.testing.assert_array_equal(got[key], np.asarray(want[key]).reshape(got[key].shape), err_msg=key)
    for key in ("pos", "seq", "slots"):
        np.testing.assert_array_equal(got[key][:n], want[key], err_msg=key)
        assert (got[key][n:] == -7).all(), f"{key}: rows behind the last token were written"
    assert got["left"][0] == want["left"] and got["status"][0] == want["status"]


def draw(B, pps, hi_len, hi_new, seed, spare=3):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, hi_len + 1, B)
    new = np.minimum(rng.integers(0, hi_new + 1, B), pps * P - lens)
    need = sum(ref.pages_of(int(a + b)) - ref.pages_of(int(a)) for a, b in zip(lens, new))
    return lens, new, rng.permutation(need + spare)


@pytest.mark.parametrize("B,pps,hi_len,hi_new", [
    (1, 1, 0, 256), (1, 3, 700, 1), (3, 2, 256, 256), (16, 33, 8192, 1), (37, 9, 2000, 300), (511, 4, 1000, 3),
    (513, 4, 1000, 3), (1025, 3, 600, 40), (5000, 2, 500, 2), (16384, 1, 200, 1)])
def test_plan_matches_the_loop(B, pps, hi_len, hi_new):
    lens, new, free = draw(B, pps, hi_len, hi_new, B)
    got, want = plan(lens, new, pps, free)
    assert want["status"] == 0
    check(got, want)


def test_page_borders():
    lens = [0, 0, 255, 256, 257, 511, 512, 1, 0]
    new = [256, 257, 1, 1, 255, 1, 0, 0, 0]
    check(*plan(lens, new, 4, np.arange(20)[::-1].copy()))


@pytest.mark.parametrize("kw", [dict(count=3), dict(count=0), dict(count=-4), dict(count=99), dict(n_cap=300), dict(n_cap=1),
                                dict(n_cap=0)])
def test_served_up_to_the_first_that_does_not_fit(kw):
    """Fewer pages or rows than asked for: what is behind the cut keeps its length, smaller requests too."""
    got, want = plan([10, 250, 0, 256, 3], [5, 300, 256, 1, 1], 4, list(range(40, 48)), **kw)
    check(got, want)


def test_invalid_sequences_are_passed_over():
    got, want = plan([-1, 5, 0, 1000, 2000000000, 7], [1, -3, 2, 25, 2000000000, 1], 4, list(range(9)), n_cap=8)
    assert want["status"] == 1 and want["cu"][-1] == 3
    check(got, want)


def test_page_ids_out_of_range_give_no_slot():
    table = np.full((3, 4), 5)
    table[0, 0], table[1, 0] = -1, 900
    got, want = plan([10, 10, 10], [300, 2, 2], 4, [1, -5, 800, 3], num_pages=800, table=table)
    assert want["status"] == 1 and (np.asarray(want["slots"]) == -1).any()
    check(got, want)


def test_unaligned_outputs():
    """Token rows that start 4 or 8 bytes off a 16-byte boundary."""
    lens, new, free = draw(9, 5, 900, 200, 5)
    n_cap = int(new.sum()) + 1
    buf = [torch.full((n_cap + 1,), -7, dtype=d, device="cuda") for d in (torch.int32, torch.int32, torch.int64)]
    o = {"table": cu32((7000 + np.arange(45)).reshape(9, 5)), "new_lens": cu32([0] * 9), "cu": cu32([0] * 10), "left": cu32([0]),
         "status": cu32([0]), "pos": buf[0][1:], "seq": buf[1][1:], "slots": buf[2][1:]}
    want = ref.page_plan(lens, new, list(free), len(free), (7000 + np.arange(45)).reshape(9, 5), 1 << 20, n_cap)
    lkv.lkv_page_plan(9, 5, 1 << 20, n_cap, cu32(lens), cu32(new), cu32(free), len(free), cu32([len(free)]), o["table"], o["new_lens"],
                      o["cu"], o["pos"], o["seq"], o["slots"], o["left"], o["status"])
    check({k: v.cpu().numpy() for k, v in o.items()}, want)
    assert all(int(x[0]) == -7 for x in buf)


def test_no_sequences():
    check(*plan([], [], 4, [1, 2]))


def test_captured_and_replayed_with_other_lengths():
    """The graph reads the lengths that stand in the buffers when it runs."""
    B, pps = 9, 5
    lens, new = cu32([0] * B), cu32([0] * B)
    free, count = cu32(np.arange(100)), cu32([100])
    table, n_cap = cu32(np.full((B, pps), -1)), 4000
    o = [cu32([-7] * B), cu32([-7] * (B + 1)), cu32([-7] * n_cap), cu32([-7] * n_cap),
         torch.full((n_cap,), -7, dtype=torch.int64, device="cuda"), cu32([-7]), cu32([-7])]
    call = lambda: lkv.lkv_page_plan(B, pps, 100, n_cap, lens, new, free, 100, count, table, *o)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (1, 2):
        a, b, _ = draw(B, pps, 900, 300, seed)
        lens.copy_(cu32(a)), new.copy_(cu32(b)), table.fill_(3), [x.fill_(-7) for x in o]
        g.replay()
        torch.cuda.synchronize()
        want = ref.page_plan(a, b, list(range(100)), 100, np.full((B, pps), 3), 100, n_cap)
        got = dict(zip(("new_lens", "cu", "pos", "seq", "slots", "left", "status"), (x.cpu().numpy() for x in o)))
        check({**got, "table": table.cpu().numpy()}, want)
