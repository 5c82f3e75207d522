"""Calls of the C entry points from several host threads at once: what one call sets up
for its launch (the shared memory that its batch needs) must not get in the way of
the other's.  Through ctypes, which lets go of the interpreter lock for the call."""
import ctypes
import threading

import pytest
import torch

from quantized_kv_cache_lkv_b200 import buffers, lkv

pytestmark = pytest.mark.gpu
K6V4 = lkv.lkv_qspec(6, 4, 64)


def statuses(*calls, times=20000):
    """The distinct statuses of each call, made `times` times from a thread of its own on a stream of its own."""
    got = [set() for _ in calls]
    start = threading.Barrier(len(calls))

    def loop(i):
        s = torch.cuda.Stream()
        start.wait()
        for k in range(times):
            got[i].add(calls[i](s.cuda_stream))
            if k % 100 == 99:
                s.synchronize()
        s.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return got


def p(t):
    return ctypes.c_void_p(t.data_ptr())


def test_attention_of_different_batches():
    keep = []

    def make(B):
        Hq, Hkv, T, D = 1, 1, 16, 64
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        q, out = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, Hq, D, device="cuda")
        c = buffers.alloc_cache(6, 4, 64, B, Hkv, T, D, zero=True)
        ws = buffers.alloc_workspace(lkv.lkv_multi_workspace_bytes(K6V4, B, Hq, Hkv, T, D, 1))
        keep.append((lens, q, out, c, ws))
        rule = lkv.lkv_score_rule(0.125)
        return lambda s: lkv.lib().lkv_decode_attention_multi(
            K6V4, B, Hq, Hkv, T, D, 1, B, p(lens), None, p(q), p(c["k_codes"]), p(c["k_sz"]), p(c["v_codes"]), p(c["v_sz"]), rule,
            p(out), None, p(ws), ws.numel(), s)

    assert statuses(make(4096), make(1), make(2000), make(1)) == [{lkv.LKV_OK}] * 4


def test_plans_of_different_batches():
    keep = []

    def make(B):
        i = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        a = dict(lens=i(B), new=i(B), free=i(1), count=i(1), table=i(B), new_lens=i(B), cu=i(B + 1), pos=i(1), seq=i(1),
                 slots=torch.zeros(1, dtype=torch.int64, device="cuda"), left=i(1), status=i(1))
        keep.append(a)
        t = {key: p(x) for key, x in a.items()}
        return lambda s: lkv.lib().lkv_page_plan(B, 1, 1, 1, t["lens"], t["new"], t["free"], 1, t["count"], t["table"], t["new_lens"],
                                                 t["cu"], t["pos"], t["seq"], t["slots"], t["left"], t["status"], s)

    assert statuses(make(16384), make(6500)) == [{lkv.LKV_OK}] * 2
