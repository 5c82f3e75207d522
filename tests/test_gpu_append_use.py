"""lkv_rope_append_kv and lkv_page_plan as serving loops use them: capacities far
above the tokens that come, one norm weight without the other, heads that the norm
or the quantizer could lose, and two batches entering one cache at once -- all bit
for bit against the formula and the oracle's quantizer."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from quantized_kv_cache_lkv_b200 import lkv
from test_gpu_rope import make, run

pytestmark = pytest.mark.gpu
G, D = 64, 128


def pool(pages, Hkv, fill=0xA5):
    """A K6V4 cache of 256-token pages."""
    return [torch.full((pages, Hkv, 256, D * 6 // 8), fill, dtype=torch.uint8, device="cuda"),
            torch.full((pages, Hkv, 256, D // G, 2), 3.5, device="cuda"),
            torch.full((pages, Hkv, 256, D * 4 // 8), fill, dtype=torch.uint8, device="cuda"),
            torch.full((pages, Hkv, 256, D // G, 2), 3.5, device="cuda")]


def append(n_tokens, slots, q, k, v, wq, wk, eps, out, cache, stream=None, pos=None, table=None):
    cap, Hq = q.shape[:2]
    lkv.lkv_rope_append_kv((6, 4, G), cap, Hq, k.shape[1], cache[0].shape[0], 256, D, n_tokens, pos, slots, q, k, v, wq, wk, eps,
                           0 if table is None else D, False, table, 0 if table is None else table.shape[0], out, *cache, stream=stream)


def expected(orc, x, Hq, Hkv, wq, wk, eps, slots, cache):
    """q_out and the cache (as `cache` held it) after rows x [n][Hq + 2 Hkv][D] went to slots, without rotation."""
    q = ref.norm_rope(x[:, :Hq], wq, eps, 0, False, None)
    k = ref.norm_rope(x[:, Hq:Hq + Hkv], wk, eps, 0, False, None)
    bits = lambda y: np.ascontiguousarray(ref.bf16_bits(y).transpose(1, 0, 2)[None])  # noqa: E731
    o = orc.quantize_kv(6, 4, G, bits(k), bits(x[:, Hq + Hkv:]), np.array([len(x)], np.int32))
    want = [t.cpu().numpy().copy() for t in cache]
    for t, s in enumerate(slots):
        for buf, key in zip(want, ("k_codes", "k_sz", "v_codes", "v_sz")):
            buf[s // 256, :, s % 256] = o[key][0, :, t].reshape(buf[s // 256, :, s % 256].shape)
    return q, want


def same(got, want, what=""):
    got = got.float().cpu().numpy() if got.dtype == torch.bfloat16 else got.cpu().numpy()
    assert np.array_equal(np.ascontiguousarray(got).view(np.uint8), np.ascontiguousarray(want).view(np.uint8)), what


def same_cache(cache, want):
    for got, w, key in zip(cache, want, ("k_codes", "k_sz", "v_codes", "v_sz")):
        same(got, w, key)


# ------------------------------------------------------------------ capacities far above the tokens
@pytest.mark.parametrize("n_tokens", [0, 1, 16, 700, -3])
@pytest.mark.parametrize("kw", [dict(D=128, rot=128), dict(D=64, rot=32), dict(D=128, rot=64, inter=True)])
def test_few_tokens_in_a_large_capacity(orc, n_tokens, kw):
    """The variant for large calls with a count far below the capacity: the rest is left as it was."""
    run(orc, N=1500, cap=1500, n_tokens=n_tokens, Hq=33, Hkv=3, G=32, seed=5 + n_tokens, **kw)


def test_rows_behind_the_count_cost_nothing():
    """16 tokens in a capacity of 16384 (32 / 8 heads of 128) take far less than the full capacity does: no row behind the
    count travels.  A full call moves 369 MB, the q, k and v rows behind the count alone would be 201 MB."""
    cap, Hq, Hkv = 16384, 32, 8
    x = torch.randn(2, cap, Hq + 2 * Hkv, D, device="cuda").to(torch.bfloat16)
    w = torch.ones(2, D, dtype=torch.bfloat16, device="cuda")
    cache, out = pool(cap // 256, Hkv), torch.empty(cap, Hq, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(cap, device="cuda")
    table = torch.rand(cap, D // 2, 2, device="cuda")
    pos = slots.to(torch.int32)

    def micros(n):
        """Device time of a call: twenty in a graph (an eager call's time is the host's), each on rows that the other
        half's have pushed out of L2."""
        count = torch.tensor([n], dtype=torch.int32, device="cuda")

        def call(i):
            y = x[i % 2]
            append(count, slots, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], w[0], w[1], 1e-6, out, cache, pos=pos, table=table)

        call(0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for i in range(20):
                call(i)
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 1e3 / 20)
        return min(times)

    few, full = micros(16), micros(cap)
    assert few < 0.2 * full, f"16 tokens {few:.1f} us, {cap} tokens {full:.1f} us"


def test_step_of_a_large_capacity_in_a_graph(orc):
    """Plan and append captured at a capacity of 16384 and replayed for steps of a few tokens: exact, and the rows behind
    the tokens stay as they were."""
    B, pps, pages, cap, Hq, Hkv = 16, 8, 160, 16384, 32, 8
    gen = torch.Generator().manual_seed(3)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mk = lambda n, dt=torch.int32: torch.full((n,), -7, dtype=dt, device="cuda")  # noqa: E731
    lens0 = [int(t) for t in torch.randint(0, 1500, (B,), generator=gen)]
    used = [-(-t // 256) for t in lens0]
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    table0 = np.full((B, pps), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table0[b, :u] = perm[at:at + u]
        at += u
    free = perm[at:].numpy()
    lens, new, table, count = i32(lens0), i32([0] * B), torch.from_numpy(table0).cuda(), i32([len(free)])
    new_lens, cu, pos, seq, slots, left, status = mk(B), mk(B + 1), mk(cap), mk(cap), mk(cap, torch.int64), mk(1), mk(1)
    x = torch.zeros(cap, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    w = (1 + 0.1 * torch.randn(2, D, generator=gen)).to(torch.bfloat16)
    wd, out, cache = w.cuda(), torch.full((cap, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda"), pool(pages, Hkv)

    def step():
        lkv.lkv_page_plan(B, pps, pages, cap, lens, new, torch_free, len(free), count, table, new_lens, cu, pos, seq, slots, left, status)
        append(cu[B:], slots, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], wd[0], wd[1], 1e-6, out, cache)

    torch_free = torch.from_numpy(free).cuda()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for news in ([1] * B, [0, 3, 0, 40] * 4):
        table.copy_(torch.from_numpy(table0))
        xs = torch.randn(cap, Hq + 2 * Hkv, D, generator=gen).to(torch.bfloat16)
        x.copy_(xs)
        new.copy_(i32(news))
        out.fill_(9.0)
        before = [t.clone() for t in cache]
        for t in (pos, seq, slots):
            t.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        want = ref.page_plan(np.array(lens0, np.int32), np.array(news, np.int32), free, len(free), table0, pages, cap)
        n = sum(news)
        assert (int(status), int(left), int(cu[B])) == (0, want["left"], n)
        assert pos[:n].tolist() == want["pos"] and seq[:n].tolist() == want["seq"] and slots[:n].tolist() == want["slots"]
        assert (pos[n:] == -7).all() and (seq[n:] == -7).all() and (slots[n:] == -7).all()
        wf = w.float().numpy()
        q, rows = expected(orc, xs[:n].float().numpy(), Hq, Hkv, wf[0], wf[1], 1e-6, want["slots"], before)
        same(out[:n], q)
        assert (out[n:] == 9.0).all()
        same_cache(cache, rows)


# ------------------------------------------------------------------ weights, values
@pytest.mark.parametrize("of_q,of_k", [(True, False), (False, True)])
@pytest.mark.parametrize("N", [3, 1500])
def test_one_weight_without_the_other(orc, of_q, of_k, N):
    """Queries normed and keys not, and the other way round, in both variants."""
    Hq, Hkv = 33, 3
    x, w, q, k, v = make(N, N, Hq, Hkv, D, N)
    wf, wd = w.float().numpy(), w.cuda()
    cache, out = pool(N // 256 + 1, Hkv), torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
    want_q, want = expected(orc, x.float().numpy(), Hq, Hkv, wf[0] if of_q else None, wf[1] if of_k else None, 1e-6, range(N), cache)
    append(None, torch.arange(N, device="cuda"), q, k, v, wd[0] if of_q else None, wd[1] if of_k else None, 1e-6, out, cache)
    same(out, want_q)
    same_cache(cache, want)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
@pytest.mark.parametrize("power", [-40, 0, 40, 60])
def test_heads_of_all_sizes(orc, eps, power):
    """Rows from 2^-40 to 2^60 through the norm and the quantizer, eps 0 among them; the largest squares pass fp32, which
    makes 0 of a row."""
    N, Hq, Hkv = 9, 6, 2
    x, w, _, _, _ = make(N, N, Hq, Hkv, D, 11, outliers=False)
    x = (x.float() * 2.0 ** power).to(torch.bfloat16)
    d, wf, wd = x.cuda(), w.float().numpy(), w.cuda()
    cache, out = pool(1, Hkv), torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([3, 200, 7, 0, 255, 8, 9, 100, 1], device="cuda")
    with np.errstate(over="ignore"):
        want_q, want = expected(orc, x.float().numpy(), Hq, Hkv, wf[0], wf[1], eps, slots.tolist(), cache)
    append(None, slots, d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], wd[0], wd[1], eps, out, cache)
    assert np.isfinite(want_q).all() and (np.abs(want_q).max() > 0 or power == 60)
    same(out, want_q)
    same_cache(cache, want)


# ------------------------------------------------------------------ streams
def test_two_batches_into_one_cache_from_two_streams(orc):
    """Each batch's rows and queries are what the formula gives, however the two calls overlap."""
    N, Hq, Hkv = 256, 4, 2
    streams = (torch.cuda.Stream(), torch.cuda.Stream())
    batches = [make(N, N, Hq, Hkv, D, 40 + i) for i in range(2)]
    outs = [torch.full((N, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = [torch.randperm(2 * N, generator=torch.Generator().manual_seed(1))[i * N:(i + 1) * N].cuda() for i in range(2)]
    weights = [w.cuda() for _, w, _, _, _ in batches]
    cache = pool(2, Hkv)
    want, want_q = cache, []
    for i, (x, w, *_) in enumerate(batches):
        wf = w.float().numpy()
        q, rows = expected(orc, x.float().numpy(), Hq, Hkv, wf[0], wf[1], 1e-6, slots[i].tolist(), want)
        want, want_q = [torch.from_numpy(r) for r in rows], want_q + [q]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            _, _, q, k, v = batches[i]
            append(None, slots[i], q, k, v, weights[i][0], weights[i][1], 1e-6, outs[i], cache, stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        same(outs[i], want_q[i])
    same_cache(cache, [t.numpy() for t in want])
