"""Sizes that the entry points' 32-bit counts cannot hold are refused by the
Python functions, not cut to their low 32 bits."""
import pytest
import torch

from fp4_weight_moe_gb300 import ops


@pytest.mark.parametrize("shape", [(2 ** 31, 1), (2 ** 32 + 1, 16), (1, 2 ** 31)])
def test_too_many_rows_or_columns(shape):
    with pytest.raises(ValueError, match="2\\^31"):
        ops._sizes(torch.empty(shape, device="meta"), "x")


def test_the_largest():
    assert tuple(ops._sizes(torch.empty(2 ** 31 - 1, 1, device="meta"), "x")) == (2 ** 31 - 1, 1)
