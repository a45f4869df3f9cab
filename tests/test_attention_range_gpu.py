"""Attention where probabilities lie far apart: a key that draws almost all of
the weight and gives nothing, as a first token's often does, leaves the output
to the many weak ones, whose share must not be lost."""
import math

import pytest
import torch

from tests.attention_exact import want
from tests.attention_util import Batch, check, check_lse, dequantise, quantise, store
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def strong_key(L, D, Hkv, G, new, above, place, seed):
    """A request whose queries of a group lie close together, with key `place` about `above` over the mean score in
    units of e, its values zero, and all other values positive."""
    b = Batch([L], D, Hkv, 64, seed)
    g = torch.Generator().manual_seed(seed + 1)
    base = torch.randn(Hkv, D, generator=g)
    q = (base.repeat_interleave(G, 0) + 0.05 * torch.randn(new, Hkv * G, D, generator=g)).to(BF16)
    for page in b.tables[0, :-(-L // 64)].tolist():  # (the signs of the values' codes)
        b.cache[page, :, :, 1, :8 * D] &= 0x77
    b.v[0] = b.v[0].abs()
    code, scale = quantise(base * (above * math.sqrt(D) / base.square().sum(-1, keepdim=True)))
    nothing = torch.zeros(D, dtype=torch.uint8)
    slot = int(b.tables[0, place // 64]) * 64 + place % 64
    for h in range(Hkv):
        store(b.cache, slot, h, 0, code[h], scale[h])
        store(b.cache, slot, h, 1, nothing, scale[h])
    b.k[0][place], b.v[0][place] = dequantise(code, scale), 0.0
    return b, q


def compare(L, D, Hkv, G, new, above, place, seed, sinks=None):
    m = _m()
    b, q = strong_key(L, D, Hkv, G, new, above, place, seed)
    out, lse = m.fp4_attention(q.cuda(), b.cache.cuda(), b.tables.cuda(), ints([L]), ints([0, new]), return_lse=True,
                               sinks=None if sinks is None else sinks.cuda())
    assert m.fp4_attention_status() == 0
    exact = want(b, q, [0, new], 1 / math.sqrt(D), sinks=sinks)
    check(out, exact[0], exact[2], above)
    check_lse(lse, exact[1], exact[3], above)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 10, 40])
@pytest.mark.parametrize("above", [12.0, 18.0, 20.0])
def test_weak_keys_beside_a_strong_one(D, new, above):
    """Groups of 4: each of the forms that 4, 12, 40 and 160 rows to a key head run in."""
    compare(8192, D, 1, 4, new, above, 0, int(above))
    compare(3000, D, 2, 4, new, above, 2900, int(above) + 7)


@pytest.mark.parametrize("new", [1, 3, 10, 40])
def test_a_very_long_context(new):
    compare(131072, 64, 1, 4, new, 18.0, 0, 3)


@pytest.mark.parametrize("new", [1, 10, 40])
def test_a_strong_sink(new):
    """The same where the sink draws the weight."""
    compare(4096, 128, 1, 4, new, 0.0, 0, 5, sinks=torch.tensor([18.0, -50.0, 3.0, 40.0]))
