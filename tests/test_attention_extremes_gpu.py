"""Attention at the ends of its inputs' ranges."""
import math

import pytest
import torch

from tests.attention_exact import want
from tests.attention_util import Batch, check, check_lse
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 10, 40])
@pytest.mark.parametrize("power", [124, 118, -112, -124])
def test_queries_near_the_ends_of_bf16(D, new, power):
    """Queries of any size that BF16 holds, where the scale brings their scores back to ordinary ones."""
    m = _m()
    b = Batch([300], D, 2, 16, 1)
    g = torch.Generator().manual_seed(new)
    q = (torch.randn(new, 8, D, generator=g) * 4).round().clamp(-15, 15) / 4  # (few bits: exact at any power)
    scale = 1 / math.sqrt(D)
    args = (b.cache.cuda(), b.tables.cuda(), ints([300]), ints([0, new]))
    big = (q.double() * 2.0 ** power).to(BF16)
    assert torch.equal(big.double(), q.double() * 2.0 ** power)
    out, lse = m.fp4_attention(big.cuda(), *args, scale=scale * 2.0 ** -power, return_lse=True)
    exact = want(b, q, [0, new], scale)
    check(out, exact[0], exact[2], power)
    check_lse(lse, exact[1], exact[3], power)
