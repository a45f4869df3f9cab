"""Norms and rotation of queries and keys, and the store into the cache of 4
bits, against the formulas in 64 bits.

Bounds of the BF16 results.  A mean of D <= 256 squares in FP32 (eight per
lane, then a tree) and rsqrt are off by less than 2^-20, the products and the
sum of the rotation by 2^-22 of their magnitudes |a c| + |b s|: 2^-19 of these
in all, and half a unit of BF16 (2^-8).  What goes into the cache is exact: the
codes of the FP32 number next to the formula's."""
import pytest
import torch

from tests.attention_util import F64, dequantise, quantise, stored
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def rotate(y, table, interleaved):
    rot = table.shape[1]
    c, s = table[:, None, :rot // 2].double(), table[:, None, rot // 2:].double()
    i = torch.arange(rot // 2)
    at, bt = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out, mag = y.clone(), y.abs()
    out[..., at] = y[..., at] * c - y[..., bt] * s
    out[..., bt] = y[..., bt] * c + y[..., at] * s
    mag[..., at] = (y[..., at] * c).abs() + (y[..., bt] * s).abs()
    mag[..., bt] = (y[..., bt] * c).abs() + (y[..., at] * s).abs()
    return out, mag


def formula(x, w, table, eps, offset, interleaved):
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (offset + w.float()).double()
    if table is None:
        return y, y.abs()
    return rotate(y, table, interleaved)


def check(got, want, mag):
    err = (got.double().cpu() - want).abs()
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -18 * mag + 2.0 ** -130
    assert (err <= bound).all(), float((err / bound).max())


def inputs(T, Hq, Hkv, D, seed, gated=False):
    g = torch.Generator().manual_seed(seed)
    wide = (2 if gated else 1) * Hq
    x = (torch.randn(T, (wide + 2 * Hkv) * D, generator=g) * 3).to(BF16).cuda()
    q = x[:, :wide * D].view(T, Hq, -1)[:, :, :D]
    k, v = x[:, wide * D:(wide + Hkv) * D].view(T, Hkv, D), x[:, (wide + Hkv) * D:].view(T, Hkv, D)
    wq, wk = (1 + 0.3 * torch.randn(D, generator=g)), (1 + 0.3 * torch.randn(D, generator=g))
    return q, k, v, wq, wk


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 32), (128, 112), (256, 256), (256, 64), (256, 48)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (3, 5, 1), (2, 32, 8), (67, 7, 7), (130, 16, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_formula(D, rot, T, Hq, Hkv, interleaved):
    m = _m()
    q, k, _, wq, wk = inputs(T, Hq, Hkv, D, D + T, gated=Hq == 16)
    table = m.rotary_table(5000, rot, device="cpu")
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(T))
    f32 = T == 67
    dtype = torch.float32 if f32 else BF16
    wq, wk = wq.to(dtype), wk.to(dtype)
    got_q, got_k = m.qk_norm_rope(q, k, pos.to(torch.int64 if f32 else torch.int32).cuda(), table.cuda(), wq.cuda(),
                                  wk.cuda(), eps=1e-5, weight_offset=1.0 if T == 3 else 0.0, interleaved=interleaved)
    for got, x, w in ((got_q, q, wq), (got_k, k, wk)):
        assert got.is_contiguous() and got.shape == x.shape
        check(got, *formula(x.cpu(), w, table[pos], 1e-5, 1.0 if T == 3 else 0.0, interleaved))


def test_parts_left_out():
    """No norm of one side, no norm at all, no rotation."""
    m = _m()
    q, k, _, wq, wk = inputs(9, 4, 2, 128, 5)
    table, pos = m.rotary_table(50, 64, device="cpu"), torch.arange(9, dtype=torch.int32)
    for w1, w2, rotary in ((wq, None, table), (None, wk, table), (None, None, table), (wq, wk, None), (None, None, None)):
        got_q, got_k = m.qk_norm_rope(q, k, pos.cuda() if rotary is not None else None,
                                      None if rotary is None else rotary.cuda(), None if w1 is None else w1.cuda(),
                                      None if w2 is None else w2.cuda())
        t = None if rotary is None else table[pos.long()]
        check(got_q, *formula(q.cpu(), w1, t, 1e-6, 0.0, False))
        check(got_k, *formula(k.cpu(), w2, t, 1e-6, 0.0, False))


@pytest.mark.parametrize("D,rot,page", [(64, 32, 16), (128, 128, 32), (128, 64, 128), (256, 64, 64), (256, 256, 16)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 2, 1), (5, 6, 3), (300, 8, 8)])
@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.37, 2.5)])
def test_store(D, rot, page, T, Hq, Hkv, scales):
    m = _m()
    q, k, v, wq, wk = inputs(T, Hq, Hkv, D, 7 * D + T)
    wq, wk = wq.to(BF16), wk.to(BF16)
    table = m.rotary_table(70000, rot, device="cpu")
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(60000, 70000, (T,), generator=g)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T]
    cache = m.alloc_fp4_cache(pages, page, Hkv, D)
    cache.fill_(0x55)
    before = cache.cpu()
    interleaved = T == 5
    got_q, none = m.qk_norm_rope(q, k, pos.to(torch.int32).cuda(), table.cuda(), wq.cuda(), wk.cuda(), v=v, cache=cache,
                                 slots=slots.cuda(), k_scale=scales[0], v_scale=scales[1], interleaved=interleaved)
    assert none is None
    check(got_q, *formula(q.cpu(), wq, table[pos], 1e-6, 0.0, interleaved))
    kf = formula(k.cpu(), wk, table[pos], float(torch.tensor(1e-6)), 0.0, interleaved)[0].float()
    by = torch.tensor(scales, dtype=torch.float32)
    want = [dequantise(*quantise(x.cpu().float() / s)) for x, s in ((kf, by[0]), (v, by[1]))]
    got = stored(cache.cpu(), slots, D)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # nothing else is written
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots] = False
    rest = torch.arange(pages * page)[rest]
    assert all(torch.equal(a, b) for a, b in zip(stored(cache.cpu(), rest, D), stored(before, rest, D)))
    # the way back: FP32 products rounded to BF16, zeros for what is no slot
    ask = torch.cat([slots, torch.tensor([-1, pages * page, 1 << 40])])
    rk, rv = m.fp4_cache_read(cache, ask.cuda(), *scales)
    assert rk.shape == (T + 3, Hkv, D) and (rk[T:] == 0).all() and (rv[T:] == 0).all()
    for r, x, s in ((rk, got[0], by[0]), (rv, got[1], by[1])):
        assert torch.equal(r[:T].cpu(), (x.float() * s).to(BF16))


def test_store_extremes():
    """Zero blocks, values past the scales' range, tiny ones, and ties of both roundings."""
    m = _m()
    D = 64
    v = torch.zeros(6, 1, D, dtype=BF16)
    v[1, 0, :16] = 5000.0
    v[2, 0, :16] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5.0, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, 0.0])
    v[3, 0] = 2.0 ** -12
    v[4, 0, ::16] = 2.0 ** -7
    v[5, 0] = torch.linspace(-6, 6, D)
    cache = m.alloc_fp4_cache(1, 16, 1, D)
    m.qk_norm_rope(v.cuda(), v.cuda(), v=v.cuda(), cache=cache, slots=torch.arange(6).cuda())
    want = dequantise(*quantise(v.float()))
    got = stored(cache.cpu(), torch.arange(6), D)
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
    assert float(got[0][1].max()) == 2688.0


def test_not_finite():
    """An infinity or a NaN of a key or a value marks that token's key in that head, and no other."""
    m = _m()
    T, H, D = 6, 3, 128
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn(T, H, D, generator=g).to(BF16), torch.randn(T, H, D, generator=g).to(BF16)
    k[1, 0, 5], k[2, 1, 100], v[3, 2, 17], v[4, 0, 127] = float("nan"), float("inf"), float("-inf"), float("nan")
    cache = m.alloc_fp4_cache(1, 16, H, D)
    m.qk_norm_rope(k.cuda(), k.cuda(), v=v.cuda(), cache=cache, slots=torch.arange(T).cuda())
    rk, rv = m.fp4_cache_read(cache, torch.arange(T).cuda())
    bad = torch.zeros(T, H, dtype=torch.bool)
    bad[1, 0] = bad[2, 1] = bad[3, 2] = bad[4, 0] = True
    assert torch.equal(rk.isnan().all(-1).cpu(), bad) and torch.equal(rk.isnan().any(-1).cpu(), bad)
    blocks = rv.isnan().view(T, H, D // 16, 16).cpu()
    assert blocks[3, 2, 1].all() and blocks[4, 0, 7].all() and int(blocks.sum()) == 32


def test_padding_and_bad_positions():
    m = _m()
    q, k, v, wq, wk = inputs(5, 2, 2, 64, 1)
    cache = m.alloc_fp4_cache(2, 16, 2, 64)
    cache.fill_(0x33)
    before = cache.clone()
    table = m.rotary_table(10, 32)
    slots = torch.tensor([-1, 32, 1 << 33, -(1 << 40), 3]).cuda()
    pos = torch.tensor([0, 1, 10, -1, 10], dtype=torch.int32).cuda()
    got, _ = m.qk_norm_rope(q, k, pos, table, wq.cuda(), wk.cuda(), v=v, cache=cache, slots=slots)
    assert got[:2].isfinite().all()
    assert got[2:, :, :32].isnan().all() and got[2:, :, 32:].isfinite().all()
    rk, _ = m.fp4_cache_read(cache, torch.tensor([3]).cuda())
    assert rk.isnan().all()
    cache[0, :, 0] = before[0, :, 0]
    assert torch.equal(cache, before)


def test_large_rows():
    """Row offsets past 32 bits."""
    m = _m()
    T, stride = 3, (1 << 31) // 2 + 64
    q = torch.empty(2 * stride + 2 * 64, dtype=BF16, device="cuda").as_strided((T, 2, 64), (stride, 64, 1))
    x = torch.randn(T, 2, 64, generator=torch.Generator().manual_seed(0)).to(BF16)
    q.copy_(x)
    got, _ = m.qk_norm_rope(q, q[:, :1])
    assert torch.equal(got.cpu(), x)


def test_refusals():
    m = _m()
    q, k, v, wq, wk = inputs(4, 4, 2, 64, 1)
    pos, table = torch.zeros(4, dtype=torch.int32, device="cuda"), m.rotary_table(10, 32)
    cache, slots = m.alloc_fp4_cache(2, 16, 2, 64), torch.arange(4, device="cuda")
    good = dict(q=q, k=k, positions=pos, rotary=table, q_weight=wq.cuda(), k_weight=wk.cuda(), v=v, cache=cache,
                slots=slots)
    m.qk_norm_rope(**good)
    for bad in (dict(q=q.float()), dict(k=k.half()), dict(rotary=table.double()), dict(q_weight=wq.cuda().half()),
                dict(q_weight=wq.to(BF16).cuda()), dict(cache=cache.float()), dict(positions=pos.float()),
                dict(slots=slots.int())):
        with pytest.raises(TypeError):
            m.qk_norm_rope(**(good | bad))
    for bad in (dict(k=k[:3]), dict(k=k[..., :32]), dict(q=q.transpose(1, 2)), dict(positions=None), dict(rotary=None),
                dict(positions=pos[:3]), dict(slots=None), dict(v=None), dict(v=v[:, :1]), dict(cache=None),
                dict(cache=m.alloc_fp4_cache(2, 16, 1, 64)), dict(cache=cache[:, :, :, :1]), dict(q=q[0]),
                dict(k_weight=wk[:32].cuda()), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            m.qk_norm_rope(**(good | bad))
    odd = torch.empty(4 * 2 * 64 + 1, dtype=BF16, device="cuda")[1:].view(4, 2, 64)
    for bad in (dict(k=odd), dict(k_scale=0.0), dict(v_scale=float("nan")), dict(eps=-1.0),
                dict(rotary=m.rotary_table(10, 24))):
        with pytest.raises(m.MoeFp4Error):
            m.qk_norm_rope(**(good | bad))
    with pytest.raises(m.MoeFp4Error):
        m.qk_norm_rope(torch.zeros(1, 1, 96, dtype=BF16, device="cuda"), torch.zeros(1, 1, 96, dtype=BF16, device="cuda"))
    with pytest.raises(m.MoeFp4Error):
        m.alloc_fp4_cache(2, 20, 2, 64)
    with pytest.raises(ValueError):
        m.fp4_cache_read(cache, slots.view(2, 2))
    with pytest.raises(TypeError):
        m.fp4_cache_read(cache, slots.int())
