"""Attention of requests that are longer than their table rows: the tokens
past them are not looked for, whatever lies in a chip's memory from before."""
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


def leave_nan(m, D, Hq, Hkv, new):
    """A call of the same form on keys and values of NaN, over more requests than there are processors."""
    R, pages = 400, 16
    cache = torch.full((pages, Hkv, 4, 2, 9 * D), 0x7f, dtype=torch.uint8, device="cuda")
    tables = (torch.arange(R * 16, device="cuda") % pages).to(torch.int32).view(R, 16)
    q = torch.ones(R * new, Hq, D, dtype=BF16, device="cuda")
    offsets = (torch.arange(R + 1, device="cuda") * new).to(torch.int32)
    assert m.fp4_attention(q, cache, tables, ints([1024] * R), offsets).isnan().all()


def compare(lengths, new, D, page, width, window=0, sinks=False, seed=0):
    m = _m()
    Hq, Hkv = 8, 2
    b = Batch(lengths, D, Hkv, page, seed)
    T, offsets = new * len(lengths), [new * i for i in range(len(lengths) + 1)]
    q = (torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(seed + 1)) * 1.5).to(BF16)
    s = torch.randn(Hq, generator=torch.Generator().manual_seed(seed + 2)) if sinks else None
    args = (q.cuda(), b.cache.cuda(), b.tables.cuda()[:, :width], ints(lengths), ints(offsets))
    more = dict(window=window, sinks=None if s is None else s.cuda(), return_lse=True)
    leave_nan(m, D, Hq, Hkv, new)
    out, lse = m.fp4_attention(*args, **more)
    exact = want(b, q, offsets, 1 / math.sqrt(D), window, s, capacity=width * page)
    check(out, exact[0], exact[2], (page, width))
    check_lse(lse, exact[1], exact[3], (page, width))
    again = m.fp4_attention(*args, **more)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert m.fp4_attention_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 5, 40])
@pytest.mark.parametrize("page,width", [(16, 1), (16, 3), (16, 8), (32, 1), (32, 5), (64, 1), (64, 3), (128, 1)])
def test_past_the_table(D, new, page, width):
    """Groups of 4 (4, 12, 20 and 160 rows to a key head); rows that end inside, at and behind the table."""
    full = width * page
    compare([full + 20, full - 1 if full > 40 else 40, 3 * full + 41], new, D, page, width, seed=full)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 5, 40])
@pytest.mark.parametrize("window", [20, 33, 70, 2 ** 31 - 1])
def test_past_the_table_under_a_window(D, new, window):
    """Windows that begin before the table's end, and some queries' behind it."""
    compare([100, 68, 47], new, D, 16, 3, window=window, sinks=window == 33, seed=window % 1000)


@pytest.mark.parametrize("new", [1, 3, 5, 40])
def test_long_requests_that_workers_share(new):
    compare([5000, 9000], new, 128, 16, 257, seed=4)
