"""What the binding makes of tensors, without a GPU: rows and their strides, pools of 4-bit records."""
from types import SimpleNamespace

import pytest
import torch

from speculative_decode_verify_attn_gb300 import vfy

CTX = SimpleNamespace(device=-1, heads=(4, 2, 64), chunk_bytes=2 * vfy.packed_bytes(64))   # (a host tensor's device number)


@pytest.mark.parametrize("stride", [256, 257, 260, 264, 1000])
@pytest.mark.parametrize("flat", [False, True])
def test_one_row_of_any_view_is_a_packed_row(stride, flat):
    wide = torch.zeros((3, stride), dtype=torch.bfloat16)
    for rows in (wide[:1], wide[2:], wide[1:1]):
        row = rows[:, :256] if flat else rows[:, :256].unflatten(1, (4, 64))
        assert vfy._rows(CTX, row, 0, "q") == (row.data_ptr(), 256)
    two = wide[:2, :256] if flat else wide[:2, :256].unflatten(1, (4, 64))
    assert vfy._rows(CTX, two, 0, "q") == (two.data_ptr(), stride)


SIZE = vfy.packed_bytes(64)


@pytest.mark.parametrize("shape,count,ok", [
    ((4, 2, SIZE), 4, True), ((4, 2, SIZE), 3, True), ((8, SIZE), 4, True), ((4, 2 * SIZE), 4, True), ((8 * SIZE,), 4, True),
    ((1, 4, 2, SIZE), 4, True), ((4, 2, SIZE), 0, True),
    ((4, 2, SIZE), 5, False),                     # fewer chunks than named
    ((4, 1, SIZE), 4, False),                     # one KV head's
    ((4, 2, SIZE // 2), 4, False), ((4, 2, 2 * SIZE), 4, False), ((4, 2, SIZE - 16), 4, False),   # another head size's records
    ((8 * SIZE - 1,), 4, False), ((0, 2, SIZE), 1, False),
])
@pytest.mark.parametrize("address", [vfy._ptr, vfy._store])
def test_pools_hold_the_records_that_are_named(shape, count, ok, address):
    t = torch.zeros(shape, dtype=torch.uint8)
    if ok:
        at = vfy._records(CTX, t, count, "k_pool", address)
        assert getattr(at, "value", at) == t.data_ptr()
    else:
        with pytest.raises(ValueError, match="k_pool"):
            vfy._records(CTX, t, count, "k_pool", address)


def test_every_packed_call_looks_at_its_pools():
    """A short pool or store among good arguments: refused before the library is called."""
    import __graft_entry__
    __graft_entry__.build()
    good, short = torch.zeros((4, 2, SIZE), dtype=torch.uint8), torch.zeros((3, 2, SIZE), dtype=torch.uint8)
    x, i = torch.zeros((1, 2, 64), dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    ctx = SimpleNamespace(device=-1, heads=(4, 2, 64), chunk_bytes=2 * SIZE, handle=None)
    calls = {"host": [lambda a, b: vfy.vfy_append_full_packed(ctx, x, x, i, i, i, i, a, b, 4, good, good, 4, 1.0, 1.0, 1, stream),
                      lambda a, b: vfy.vfy_page_in_packed(ctx, a, b, 4, good, good, 4, i, i, 1, 1, stream)],
             "pool": [lambda a, b: vfy.vfy_append_full_packed(ctx, x, x, i, i, i, i, good, good, 4, a, b, 4, 1.0, 1.0, 1, stream),
                      lambda a, b: vfy.vfy_page_in_packed(ctx, good, good, 4, a, b, 4, i, i, 1, 1, stream),
                      lambda a, b: vfy.vfy_unpack_chunks(ctx, a, b, 4, i, 1, 1.0, 1.0, x, x, stream),
                      lambda a, b: vfy.vfy_attend_full_packed(ctx, x, i, a, b, 4, i, i, i, 1, i, 1.0, 1.0, x, None, 1, stream)]}
    stream = SimpleNamespace(cuda_stream=0)
    for kind, some in calls.items():
        for call in some:
            for a, b, name in ((short, good, "k"), (good, short, "v")):
                with pytest.raises(ValueError, match=f"host_{name}" if kind == "host" else f"{name}_pool"):
                    call(a, b)


def test_no_store_is_no_address():
    assert vfy._store(CTX, None, vfy.U8, "host_k") is None       # the library refuses it
    with pytest.raises(TypeError):
        vfy._store(CTX, [1, 2], vfy.U8, "host_k")
