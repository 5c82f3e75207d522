"""What the native binding refuses of tensors on a GPU -- type, room, layout --
and streams given as torch streams and as handles."""
import pytest
import torch

from quantized_kv_cache_lkv_b200 import lkv

pytestmark = pytest.mark.gpu


def table(t, rows=8, spec=None, stream=None):
    lkv.lkv_rope_table(spec or lkv.lkv_rope_spec("none", 32), rows, t, stream=stream)


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(8, 16, 2, device="cuda", dtype=torch.float64),   # another type
    lambda: torch.zeros(7, 16, 2, device="cuda"),                        # a row short
    lambda: torch.zeros(16, 16, 2, device="cuda")[::2],                  # rows apart
    lambda: torch.zeros(8, 2, 16, device="cuda").transpose(1, 2),        # another order
    lambda: torch.zeros(8, 16, 2),                                       # on the host
])
def test_tensors_that_do_not_fit(make):
    with pytest.raises(lkv.LkvError) as e:
        table(make())
    assert e.value.status == lkv.LKV_ERR_INVALID_ARG and "lkv_rope_table" in str(e.value)


def test_views_of_a_projection():
    """Heads of a token have to lie side by side; tokens may lie apart."""
    x = torch.zeros(4, 12, 128, device="cuda", dtype=torch.bfloat16)
    out = torch.zeros(4, 4, 128, device="cuda", dtype=torch.bfloat16)
    c = [torch.zeros(1, 4, 256, 96, dtype=torch.uint8, device="cuda"), torch.zeros(1, 4, 256, 2, 2, device="cuda"),
         torch.zeros(1, 4, 256, 64, dtype=torch.uint8, device="cuda"), torch.zeros(1, 4, 256, 2, 2, device="cuda")]
    slots = torch.arange(4, device="cuda")

    def call(q, k=x[:, 4:8], v=x[:, 8:]):
        lkv.lkv_rope_append_kv((6, 4, 64), 4, 4, 4, 1, 256, 128, None, None, slots, q, k, v, None, None, 0.0, 0, False, None, 0, out, *c)
        torch.cuda.synchronize()

    call(x[:, :4])
    for bad in (x[:, :8:2], x[:3, :4], x[:, :3], x[:, :4].float(), x[:, :4, :64], x.transpose(0, 1)[:4, :4]):
        with pytest.raises(lkv.LkvError) as e:
            call(bad)
        assert e.value.status == lkv.LKV_ERR_INVALID_ARG


def test_streams():
    """None is torch's current stream; a torch stream and a handle name their own."""
    s = torch.cuda.Stream()
    want = torch.zeros(8, 16, 2, device="cuda")
    table(want)
    torch.cuda.synchronize()
    for given in (s, s.cuda_stream, None):
        t = torch.zeros(8, 16, 2, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            table(t, stream=given)
        s.synchronize()
        assert torch.equal(t, want)


def test_sizes_past_64_bits():
    """No tensor has room for a pool whose size passes 64 bits, whatever the product's low bits are."""
    c = [torch.zeros(1, 4, 256, 96, dtype=torch.uint8, device="cuda"), torch.zeros(1, 4, 256, 2, 2, device="cuda"),
         torch.zeros(1, 4, 256, 64, dtype=torch.uint8, device="cuda"), torch.zeros(1, 4, 256, 2, 2, device="cuda")]

    def call(pages, heads):  # no tokens: nothing is launched
        lkv.lkv_rope_append_kv((6, 4, 64), 0, heads, heads, pages, 256, 128, None, None, None, None, None, None, None, None, 0.0,
                               0, False, None, 0, None, *c)

    call(1, 4)
    with pytest.raises(lkv.LkvError) as e:
        call(1 << 30, 1 << 20)
    assert e.value.status == lkv.LKV_ERR_INVALID_ARG
