"""Norms, rotation and store of so many tokens that a warp takes all heads of a
kind of its token (16 tokens to a processor and more): against the formulas in
64 bits, the stored codes exactly, and against the same tokens a few at a time."""
import pytest
import torch

from tests.attention_util import dequantise, quantise, stored
from tests.gpu_util import ensure_built
from tests.test_qk_norm_rope_gpu import check, formula, inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = float(torch.tensor(1e-6))


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def many():
    return 16 * torch.cuda.get_device_properties(0).multi_processor_count + 37


def case(D, rot, Hq, Hkv, normed, seed):
    T = many()
    q, k, v, wq, wk = inputs(T, Hq, Hkv, D, seed, gated=seed % 2 == 1)
    table = None if rot == 0 else torch.randn(3000, rot, generator=torch.Generator().manual_seed(seed))
    pos = torch.randint(0, 3000, (T,), generator=torch.Generator().manual_seed(seed + 1), dtype=torch.int32)
    return T, q, k, v, (wq.to(BF16), wk.to(BF16)) if normed else (None, None), table, pos


def call(m, q, k, w, table, pos, lo, hi, interleaved, **more):
    more = {a: (b[lo:hi] if a in ("v", "slots") else b) for a, b in more.items()}
    return m.qk_norm_rope(q[lo:hi], k[lo:hi], None if table is None else pos[lo:hi].cuda(),
                          None if table is None else table.cuda(), *(None if x is None else x.cuda() for x in w),
                          interleaved=interleaved, **more)


# (odd numbers of heads, and more key heads than one task of 32 rounds takes)
HEADS = [(64, 64, 9, 5), (64, 16, 3, 3), (64, 32, 4, 131), (128, 128, 12, 8), (128, 64, 7, 3), (128, 0, 5, 67),
         (256, 256, 5, 5), (256, 64, 3, 35)]


@pytest.mark.parametrize("D,rot,Hq,Hkv", HEADS)
@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens(D, rot, Hq, Hkv, normed, interleaved):
    m = _m()
    T, q, k, _, w, table, pos = case(D, rot, Hq, Hkv, normed, D + Hkv)
    got = call(m, q, k, w, table, pos, 0, T, interleaved)
    for y, x, ww in zip(got, (q, k), w):
        check(y, *formula(x.cpu(), ww, None if table is None else table[pos.long()], EPS, 0.0, interleaved))
    for lo in range(0, T, 1000):
        part = call(m, q, k, w, table, pos, lo, min(lo + 1000, T), interleaved)
        assert torch.equal(part[0], got[0][lo:lo + 1000]) and torch.equal(part[1], got[1][lo:lo + 1000])


@pytest.mark.parametrize("D,rot,Hq,Hkv", HEADS)
@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.37, 2.5)])
def test_many_tokens_stored(D, rot, Hq, Hkv, normed, scales):
    m = _m()
    interleaved = scales[0] != 1.0
    T, q, k, v, w, table, pos = case(D, rot, Hq, Hkv, normed, D + Hkv + 1)
    page, g = 32, torch.Generator().manual_seed(3)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::97] = -1
    caches = [m.alloc_fp4_cache(pages, page, Hkv, D).fill_(0x55) for _ in range(2)]
    before = caches[0].cpu()
    more = dict(v=v, slots=slots.cuda(), k_scale=scales[0], v_scale=scales[1])
    got_q, none = call(m, q, k, w, table, pos, 0, T, interleaved, cache=caches[0], **more)
    assert none is None
    angles = None if table is None else table[pos.long()]
    check(got_q, *formula(q.cpu(), w[0], angles, EPS, 0.0, interleaved))
    kf = formula(k.cpu(), w[1], angles, EPS, 0.0, interleaved)[0].float()
    by = torch.tensor(scales, dtype=torch.float32)
    kept = slots >= 0
    got = stored(caches[0].cpu(), slots[kept], D)
    for y, x, s in zip(got, (kf, v.cpu().float()), by):
        assert torch.equal(y, dequantise(*quantise(x[kept] / s)))
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots[kept]] = False
    rest = torch.arange(pages * page)[rest]
    assert all(torch.equal(a, b) for a, b in zip(stored(caches[0].cpu(), rest, D), stored(before, rest, D)))
    for lo in range(0, T, 1000):
        call(m, q, k, w, table, pos, lo, min(lo + 1000, T), interleaved, cache=caches[1], **more)
    assert torch.equal(*caches)


def test_not_finite_of_many_tokens():
    """An infinity or a NaN marks its token's key in its head, in whichever round of a warp's it lies."""
    m = _m()
    H, D = 11, 128
    T, _, k, v, w, _, _ = case(D, 0, 1, H, True, 4)
    k, v = k.clone(), v.clone()
    bad = torch.zeros(T, H, dtype=torch.bool)
    g = torch.Generator().manual_seed(2)
    for i in range(40):
        t, h, c = (int(torch.randint(0, n, (1,), generator=g)) for n in (T, H, D))
        (k if i % 2 else v)[t, h, c] = float("nan") if i % 3 else float("-inf")
        bad[t, h] = True
    cache = m.alloc_fp4_cache(-(-T // 16), 16, H, D)
    slots = torch.arange(T, device="cuda")
    m.qk_norm_rope(k[:, :1], k, None, None, *(x.cuda() for x in w), v=v, cache=cache, slots=slots)
    rk, _ = m.fp4_cache_read(cache, slots)
    assert torch.equal(rk.isnan().all(-1).cpu(), bad) and torch.equal(rk.isnan().any(-1).cpu(), bad)


@pytest.mark.parametrize("power", [-39, -20, 20, 46])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_stored_keys_far_from_one(D, power):
    """The norm takes a key's size away, without eps too: within the range that is stated, to the last code."""
    m = _m()
    T, Hkv = 500, 3
    q, k, v, wq, wk = inputs(T, 2, Hkv, D, 9 + D)
    k = (k.double() * 2.0 ** power).to(BF16)
    table, pos = m.rotary_table(600, D, device="cpu"), torch.arange(T, dtype=torch.int32)
    cache, slots = m.alloc_fp4_cache(T // 16 + 1, 16, Hkv, D), torch.arange(T)
    m.qk_norm_rope(q, k, pos.cuda(), table.cuda(), wq.to(BF16).cuda(), wk.to(BF16).cuda(), eps=0.0, v=v, cache=cache,
                   slots=slots.cuda())
    kf = formula(k.cpu(), wk.to(BF16), table[:T], 0.0, 0.0, False)[0].float()
    assert torch.equal(stored(cache.cpu(), slots, D)[0], dequantise(*quantise(kf)))
