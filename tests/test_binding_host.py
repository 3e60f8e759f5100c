"""What the binding makes of tensors, without a GPU: rows and their strides."""
from types import SimpleNamespace

import pytest
import torch

from speculative_decode_verify_attn_gb300 import vfy

CTX = SimpleNamespace(device=-1, heads=(4, 2, 64))              # (a host tensor's device number)


@pytest.mark.parametrize("stride", [256, 257, 260, 264, 1000])
@pytest.mark.parametrize("flat", [False, True])
def test_one_row_of_any_view_is_a_packed_row(stride, flat):
    wide = torch.zeros((3, stride), dtype=torch.bfloat16)
    for rows in (wide[:1], wide[2:], wide[1:1]):
        row = rows[:, :256] if flat else rows[:, :256].unflatten(1, (4, 64))
        assert vfy._rows(CTX, row, 0, "q") == (row.data_ptr(), 256)
    two = wide[:2, :256] if flat else wide[:2, :256].unflatten(1, (4, 64))
    assert vfy._rows(CTX, two, 0, "q") == (two.data_ptr(), stride)
