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


def all_keys_negative(b, r, h, column):
    """Key head h's codes of a column of request r: all -1 (code 10) under the scales that are there, none of them 0."""
    for page in b.tables[r, :-(-b.lengths[r] // b.page_size)].tolist():
        for block in b.cache[page, h, :, 0]:
            codes = block[:8 * b.D].view(16, b.D // 2)
            codes[:, column // 2] = (codes[:, column // 2] & (0x0f if column % 2 else 0xf0)) | (0xa0 if column % 2 else 0x0a)
            scales = block[8 * b.D:].view(16, b.D // 16)
            scales[:, column // 16] = 0x38  # (1)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,length", [(1, 1), (1, 200), (3, 90), (10, 90), (40, 300), (1, 9000), (10, 9000), (40, 9000)])
@pytest.mark.parametrize("sinks", [False, True])
def test_scores_of_minus_infinity(D, new, length, sinks):
    """A query whose scores are all -inf sees keys: 0 / 0, or, with a sink, 0; beside one that sees none."""
    m = _m()
    column = 37
    b = Batch([length, 1], D, 2, 16, 2)
    all_keys_negative(b, 0, 1, column)
    q = torch.randn(new + 2, 8, D, generator=torch.Generator().manual_seed(3)).to(BF16)
    q[:new, 6, column] = math.inf
    s = torch.randn(8, generator=torch.Generator().manual_seed(4)) if sinks else None
    out, lse = m.fp4_attention(q.cuda(), b.cache.cuda(), b.tables.cuda(), ints([length, 1]), ints([0, new, new + 2]),
                               return_lse=True, sinks=None if s is None else s.cuda())
    out, lse = out.float().cpu(), lse.cpu()
    assert torch.equal(lse[:new, 6], torch.full((new,), float(s[6]) if sinks else -math.inf))
    assert (out[:new, 6] == 0).all() if sinks else out[:new, 6].isnan().all()
    others = torch.ones(new + 2, 8, dtype=torch.bool)
    others[:new, 6] = False
    assert out[others].isfinite().all()
    assert (out[new] == 0).all() and torch.equal(lse[new], s if sinks else torch.full((8,), -math.inf))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,length", [(1, 100), (3, 90), (10, 90), (40, 300), (1, 9000), (40, 9000)])
def test_sinks_without_end(D, new, length):
    """A sink of inf takes all of the weight; one of -inf none."""
    m = _m()
    b = Batch([length], D, 2, 16, 2)
    q = torch.randn(new, 8, D, generator=torch.Generator().manual_seed(3)).to(BF16)
    args = (q.cuda(), b.cache.cuda(), b.tables.cuda(), ints([length]), ints([0, new]))
    s = torch.tensor([math.inf, -math.inf, 0.0, math.inf] * 2, device="cuda")
    out, lse = m.fp4_attention(*args, sinks=s, return_lse=True)
    plain, plain_lse = m.fp4_attention(*args, return_lse=True)
    assert (out[:, [0, 3, 4, 7]] == 0).all() and (lse[:, [0, 3, 4, 7]] == math.inf).all()
    assert torch.equal(out[:, [1, 5]], plain[:, [1, 5]]) and torch.equal(lse[:, [1, 5]], plain_lse[:, [1, 5]])
    s[0] = 3e38  # (in units of log 2 past FP32)
    out, lse = m.fp4_attention(*args, sinks=s, return_lse=True)
    assert (out[:, 0] == 0).all() and (lse[:, 0] == s[0]).all()
    bad = q.clone()
    bad[0, 0, 3] = math.nan
    out, lse = m.fp4_attention(bad.cuda(), *args[1:], sinks=s, return_lse=True)
    assert out[0, 0].isnan().all() and lse[0, 0].isnan() and (out[:, 3] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 10, 40])
@pytest.mark.parametrize("scale", [1e4, -1e6, 1e8, 1e15, 1e30])
def test_scores_far_apart(D, new, scale):
    """Scores so large that one key has all of the weight, and that a unit of FP32 at theirs is many powers of two."""
    m = _m()
    L = 500
    b = Batch([L], D, 2, 16, 3)
    q = torch.randn(new, 8, D, generator=torch.Generator().manual_seed(4)).to(BF16)
    out, lse = m.fp4_attention(q.cuda(), b.cache.cuda(), b.tables.cuda(), ints([L]), ints([0, new]), scale=scale,
                               return_lse=True)
    out, lse = out.double().cpu(), lse.double().cpu()
    sees = torch.arange(L) <= torch.arange(new)[:, None] + (L - new)
    clear = 0
    for h in range(8):
        k, v = b.k[0][:, h // 4], b.v[0][:, h // 4]
        x = (q[:, h].double() @ k.T * scale).masked_fill(~sees, -math.inf)
        off = 2.0 ** -18 * float(((q[:, h].double().abs() @ k.abs().T) * abs(scale)).max())
        top = x.topk(2, 1)
        # (where the second lies below by more than both may be off by, and by 20 besides: e^-20 of its value)
        first = top.values[:, 0] - top.values[:, 1] > 2 * off + 20
        want = v[top.indices[:, 0]]
        assert ((out[:, h] - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * v.abs().max())[first].all()
        assert ((lse[:, h] - top.values[:, 0]).abs() <= off + 2.0 ** -20 * top.values[:, 0].abs())[first].all()
        clear += int(first.sum())
    assert clear >= 4 * new
