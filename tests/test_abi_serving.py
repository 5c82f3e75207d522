"""The serving-step calls without a GPU: host-side refusals with their status
(fake device addresses are never dereferenced), calls that have nothing to do,
workspace sizes, and tensors that do not fit."""
import ctypes

import pytest
import torch

from quantized_kv_cache_lkv_b200 import lkv

FAKE = 0x7F0000000000
K6V4 = (6, 4, 64)
ARG, UNSUPPORTED, WORKSPACE = lkv.LKV_ERR_INVALID_ARG, lkv.LKV_ERR_UNSUPPORTED, lkv.LKV_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_kv_cache_lkv_b200 import build
    build.build()


def rc_of(fn, **kw):
    try:
        fn(**kw)
    except lkv.LkvError as e:
        return e.status
    return 0


def at(i):
    """Addresses 1 MiB apart, so that no two tensors overlap."""
    return FAKE + (i << 20)


def plan_args(**kw):
    a = dict(B=4, pages_per_seq=8, num_pages=64, n_cap=32, seq_lens=at(0), n_new=at(1), free_pages=at(2), free_cap=16,
             free_count=at(3), block_table=at(4), new_lens=at(5), cu_new=at(6), positions=at(7), token_seq=at(8), slots=at(9),
             free_left=at(10), status=at(11), stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), ARG), (dict(n_cap=-1), ARG), (dict(free_cap=-1), ARG), (dict(pages_per_seq=0), ARG), (dict(num_pages=0), ARG),
    (dict(B=16385), UNSUPPORTED), (dict(n_cap=(1 << 30) + 1), UNSUPPORTED), (dict(pages_per_seq=(1 << 22) + 1), UNSUPPORTED),
    (dict(seq_lens=None), ARG), (dict(n_new=None), ARG), (dict(free_pages=None), ARG), (dict(free_count=None), ARG),
    (dict(block_table=None), ARG), (dict(new_lens=None), ARG), (dict(cu_new=None), ARG), (dict(positions=None), ARG),
    (dict(token_seq=None), ARG), (dict(slots=None), ARG), (dict(free_left=None), ARG),
    (dict(slots=at(9) + 4), ARG), (dict(seq_lens=at(0) + 2), ARG), (dict(status=at(11) + 1), ARG),
    # an output on an input, or on another output
    (dict(new_lens=at(0)), ARG), (dict(new_lens=at(0) + 12), ARG), (dict(free_left=at(3)), ARG), (dict(block_table=at(2)), ARG),
    (dict(token_seq=at(7) + 124), ARG), (dict(status=at(10)), ARG), (dict(cu_new=at(5) + 12), ARG),
])
def test_plan_refuses(kw, want):
    assert rc_of(lkv.lkv_page_plan, **plan_args(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(kind=4), UNSUPPORTED), (dict(kind=-1), UNSUPPORTED), (dict(rot_dim=0), UNSUPPORTED), (dict(rot_dim=24), UNSUPPORTED),
    (dict(rot_dim=144), UNSUPPORTED), (dict(base=1.0), ARG), (dict(base=float("nan")), ARG), (dict(attn_factor=float("inf")), ARG),
    (dict(kind="linear", factor=0.0), ARG), (dict(kind="smooth", low=4.0, high=4.0), ARG), (dict(kind="ramp", low=0.0), ARG),
    (dict(kind="ramp", orig_ctx=0.0), ARG), (dict(kind="smooth", factor=float("nan")), ARG),
])
def test_table_refuses(kw, want):
    assert rc_of(lkv.lkv_rope_table, spec=lkv.lkv_rope_spec(**kw), rows=10, table=FAKE, stream=0) == want


def test_table_refuses_rows_and_address():
    ok = lkv.lkv_rope_spec()
    assert rc_of(lkv.lkv_rope_table, spec=ok, rows=-1, table=FAKE, stream=0) == ARG
    assert rc_of(lkv.lkv_rope_table, spec=ok, rows=1, table=FAKE + 8, stream=0) == ARG
    assert rc_of(lkv.lkv_rope_table, spec=ok, rows=1, table=None, stream=0) == ARG
    assert rc_of(lkv.lkv_rope_table, spec=ok, rows=0, table=None, stream=0) == 0


def append_args(**kw):
    a = dict(spec=K6V4, n_cap=8, Hq=8, Hkv=2, num_pages=4, page_tokens=256, D=128, n_tokens=at(0), positions=at(1), slots=at(2),
             q=at(3), k=at(4), v=at(5), q_weight=at(6), k_weight=at(7), eps=1e-6, rot_dim=128, interleaved=False, table=at(8),
             table_rows=16, q_out=at(9), k_codes=at(10), k_sz=at(11), v_codes=at(12), v_sz=at(13), stream=0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(spec=(5, 4, 64)), UNSUPPORTED), (dict(spec=(6, 4, 48)), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=64, spec=(6, 4, 128)), UNSUPPORTED),
    (dict(spec=(6, 4, 128), page_tokens=255), UNSUPPORTED), (dict(rot_dim=8), UNSUPPORTED), (dict(rot_dim=136), UNSUPPORTED),
    (dict(rot_dim=144), UNSUPPORTED), (dict(rot_dim=-16), UNSUPPORTED), (dict(n_cap=-1), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG),
    (dict(num_pages=0), ARG), (dict(page_tokens=0), ARG), (dict(table_rows=-1), ARG), (dict(interleaved=2), ARG), (dict(reciprocal=2), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(positions=None), ARG), (dict(slots=None), ARG), (dict(slots=at(2) + 4), ARG),
    (dict(q=None), ARG), (dict(k=at(4) + 8), ARG), (dict(v=None), ARG), (dict(q_out=None), ARG), (dict(table=None), ARG), (dict(k_codes=None), ARG),
    (dict(k_sz=None), ARG), (dict(v_sz=at(13) + 8), ARG), (dict(q_weight=at(6) + 2), ARG),
    (dict(q_stride=1016), ARG), (dict(k_stride=257), ARG), (dict(v_stride=260), ARG),
    # q_out on the rows that are read: in place, or inside a fused projection
    (dict(q_out=at(3)), ARG), (dict(q_out=at(4) + 512), ARG), (dict(q_out=at(5) - 16), ARG), (dict(q=at(9) - 8 * 1536 * 2 + 2048, q_stride=1536), ARG),
])
def test_append_refuses(kw, want):
    assert rc_of(lkv.lkv_rope_append_kv, **append_args(**kw)) == want


def multi_args(**kw):
    a = dict(spec=K6V4, B=2, Hq=8, Hkv=2, T_cap=64, D=128, max_q=4, n_rows=8, seq_lens=at(0), cu_q=at(1), q=at(2), k_codes=at(3),
             k_sz=at(4), v_codes=at(5), v_sz=at(6), rule=lkv.lkv_score_rule(0.088), out=at(7), lse=at(8), workspace=at(9),
             ws_bytes=1 << 40, stream=0)
    a.update(kw)
    return a


def rule(**kw):
    return lkv.lkv_score_rule(**{"softmax_scale": 0.1, **kw})


MULTI = [
    (dict(spec=(6, 3, 64)), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(Hq=7), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(B=-1), ARG),
    (dict(Hq=130), UNSUPPORTED), (dict(max_q=0), ARG), (dict(max_q=65), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(n_rows=-1), ARG),
    (dict(cu_q=None, n_rows=1), ARG), (dict(rule=rule(softmax_scale=float("inf"))), ARG), (dict(rule=rule(softcap=-1.0)), ARG),
    (dict(rule=rule(softcap=float("nan"))), ARG), (dict(rule=rule(softcap=1e-31)), ARG), (dict(rule=rule(window=-1)), ARG), (dict(rule=rule(slopes=FAKE + 2)), ARG),
    (dict(rule=rule(prefix_lens=FAKE + 1)), ARG), (dict(rule=rule(doc_starts=FAKE + 3)), ARG), (dict(seq_lens=None), ARG), (dict(q=None), ARG),
    (dict(q=at(2) + 8), ARG), (dict(out=None), ARG), (dict(lse=at(8) + 2), ARG), (dict(k_codes=None), ARG), (dict(k_sz=None), ARG),
    (dict(v_codes=at(5) + 4), ARG), (dict(v_sz=None), ARG), (dict(cu_q=at(1) + 2), ARG), (dict(workspace=None), ARG), (dict(workspace=at(9) + 128), ARG),
    (dict(ws_bytes=1024), WORKSPACE),
]


@pytest.mark.parametrize("kw,want", MULTI + [(dict(T_cap=(1 << 30) + 2), UNSUPPORTED), (dict(spec=(6, 4, 128), T_cap=63), UNSUPPORTED),
                                             (dict(B=4096, Hq=512, Hkv=128, T_cap=1 << 20, n_rows=1 << 20), UNSUPPORTED)])
def test_multi_refuses(kw, want):
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(**kw)) == want


@pytest.mark.parametrize("kw,want", MULTI + [(dict(pages_per_seq=0), ARG), (dict(num_pages=0), ARG), (dict(block_table=None), ARG),
                                             (dict(block_table=at(10) + 2), ARG), (dict(pages_per_seq=(1 << 22) + 1), UNSUPPORTED)])
def test_multi_paged_refuses(kw, want):
    a = multi_args(pages_per_seq=4, num_pages=9, block_table=at(10))
    for old, new in (("k_codes", "k_pool"), ("k_sz", "k_sz_pool"), ("v_codes", "v_pool"), ("v_sz", "v_sz_pool")):
        a[new] = kw.get(old, a.pop(old))
    del a["T_cap"]
    a.update({k: v for k, v in kw.items() if k in a})
    assert rc_of(lkv.lkv_decode_attention_multi_paged, **a) == want


def test_nothing_to_do():
    """Succeeds without touching a pointer or the GPU."""
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(B=0, n_rows=0, seq_lens=None, q=None, out=None, k_codes=None, k_sz=None,
                                                             v_codes=None, v_sz=None)) == 0
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(n_rows=0, q=None, out=None)) == 0
    assert rc_of(lkv.lkv_rope_append_kv, **append_args(n_cap=0, q=None, k=None, v=None, q_out=None, slots=None, positions=None)) == 0


def test_workspace_sizes():
    n = lkv.lkv_multi_workspace_bytes(K6V4, 16, 32, 8, 8192, 128, 1)
    assert 0 < n < 64 << 20 and n % 256 == 0
    # it depends on the rows of a block and the widths, not on batch or length
    assert n == lkv.lkv_multi_workspace_bytes(K6V4, 1, 32, 8, 64, 128, 2)
    assert lkv.lkv_multi_workspace_bytes(K6V4, 16, 32, 8, 8192, 128, 64) >= n
    for bad in ((K6V4, 16, 30, 8, 8192, 128, 1), ((5, 4, 64), 16, 32, 8, 8192, 128, 1), (K6V4, 16, 32, 8, 8192, 96, 1), (K6V4, 16, 32, 8, 8192, 128, 0)):
        assert lkv.lkv_multi_workspace_bytes(*bad) == 0


def test_structures_match_the_header():
    assert ctypes.sizeof(lkv.lkv_rope_spec) == 56 and ctypes.sizeof(lkv.lkv_score_rule) == 40
    s = lkv.lkv_rope_spec("ramp", 64, 500000.0, 8.0, 1.0, 4.0, 8192.0, 1.5)
    assert (s.kind, s.rot_dim, s.base, s.factor, s.low, s.high, s.orig_ctx, s.attn_factor) == (3, 64, 500000.0, 8.0, 1.0, 4.0, 8192.0, 1.5)
    with pytest.raises((TypeError, KeyError)):
        lkv.lkv_rope_spec("no such kind")


def test_tensors_that_do_not_fit():
    """Refused before an address is passed on: here for their device, as there is none to be on."""
    i = torch.zeros(64, dtype=torch.int32)
    assert rc_of(lkv.lkv_page_plan, **plan_args(seq_lens=i)) == ARG
    assert rc_of(lkv.lkv_rope_table, spec=lkv.lkv_rope_spec(), rows=1, table=torch.zeros(128), stream=0) == ARG
    assert rc_of(lkv.lkv_rope_append_kv, **append_args(q=torch.zeros(8, 8, 128, dtype=torch.bfloat16))) == ARG
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(rule=rule(slopes=torch.zeros(8)))) == ARG
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(workspace=torch.zeros(1 << 20, dtype=torch.uint8), ws_bytes=1 << 20)) == ARG
    with pytest.raises(TypeError):
        lkv.lkv_page_plan(**plan_args(seq_lens="lens"))
    with pytest.raises(TypeError):
        lkv.lkv_decode_attention_multi(**multi_args(rule=None))
    with pytest.raises(OverflowError):
        lkv.lkv_page_plan(**plan_args(B=1 << 40))


def test_arguments_by_position_and_name():
    """Both reach the same call; a name that is unknown, given twice or missing is refused."""
    ok = lkv.lkv_rope_spec()
    assert rc_of(lkv.lkv_rope_table, stream=0, table=FAKE + 8, rows=1, spec=ok) == ARG
    with pytest.raises(lkv.LkvError) as e:
        lkv.lkv_rope_table(ok, 1, FAKE + 8, stream=0)
    assert e.value.status == ARG
    assert lkv.lkv_rope_table(ok, 0, None, 0) is None
    for args, kw in (((ok, 0, None, 0, 0), {}), ((ok, 0), {}), ((ok, 0, None), dict(row=1)), ((ok, 0, None), dict(rows=1)), ((), {})):
        with pytest.raises(TypeError):
            lkv.lkv_rope_table(*args, **kw)


@pytest.mark.parametrize("spec,want", [((6, 4, 64), 0), ([6, 4, 64], 0), (lkv.lkv_qspec(6, 4, 64), 0), ((5, 4, 64), lkv.LKV_ERR_UNSUPPORTED)])
def test_spec_forms(spec, want):
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(spec=spec, n_rows=0, q=None, out=None)) == want


@pytest.mark.parametrize("spec", [(6, 4), None, "k6v4", (6, 4, "64"), lkv.lkv_rope_spec()])
def test_specs_refused(spec):
    with pytest.raises(TypeError):
        lkv.lkv_decode_attention_multi(**multi_args(spec=spec))


@pytest.mark.parametrize("flag,want", [(None, 0), (False, 0), (True, 0), (0, 0), (1, 0), (2, ARG), (-1, ARG)])
def test_reciprocal_is_a_flag(flag, want):
    assert rc_of(lkv.lkv_rope_append_kv, **append_args(n_cap=0, q=None, k=None, v=None, q_out=None, slots=None, positions=None,
                                                       reciprocal=flag)) == want


@pytest.mark.parametrize("scale,cap,want", [(1e38, 1e-3, ARG), (-1e38, 1e-3, ARG), (3e38, 0.0, ARG), (3e38, 50.0, 0), (2e38, 0.0, 0),
                                            (1e-38, 1e-30, 0)])
def test_score_factor_is_finite(scale, cap, want):
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(rule=rule(softmax_scale=scale, softcap=cap), n_rows=0, q=None, out=None)) == want


@pytest.mark.parametrize("scale,cap,want", [(0.1, 3.4e38, 0), (1e38, 1e31, 0), (2e38, 3e38, 0), (3e38, 3e38, ARG), (3e38, 1e30, 0)])
def test_caps_above_1e30_are_none(scale, cap, want):
    """Such a cap is accepted; the factor of the scores is then the scale itself."""
    assert rc_of(lkv.lkv_decode_attention_multi, **multi_args(rule=rule(softmax_scale=scale, softcap=cap), n_rows=0, q=None, out=None)) == want


@pytest.mark.parametrize("ws", [at(9), torch.zeros(64, dtype=torch.uint8), None])
@pytest.mark.parametrize("size", [-1, -256, -(1 << 63)])
def test_negative_workspace_size(ws, size):
    """Not taken for 2^64 less as much, which any workspace would seem to have room for.  Nothing is launched here (no rows)."""
    a = multi_args(workspace=ws, ws_bytes=size, n_rows=0, q=None, out=None)
    assert rc_of(lkv.lkv_decode_attention_multi, **a) == ARG
    a.update(pages_per_seq=4, num_pages=9, block_table=at(10))
    for old, new in (("k_codes", "k_pool"), ("k_sz", "k_sz_pool"), ("v_codes", "v_pool"), ("v_sz", "v_sz_pool")):
        a[new] = a.pop(old)
    del a["T_cap"]
    assert rc_of(lkv.lkv_decode_attention_multi_paged, **a) == ARG
