"""The norms before and after a block with its gate and residual scale,
against the definition in 64 bits.

Bounds.  A mean of H squares in FP32, summed by threads of at most 32 values
and a tree, is off by less than 2^-17 of itself and rsqrt by 2 units, so a
norm factor is off by less than 2^-17; the products and the sum after it by
2^-22 of their magnitudes.  With t = |scale gate z|: |dr'| <= 2^-16 t +
2^-22 |r|, and |dn| <= 2^-16 |n| + |n / r'| |dr'| plus the share of dr' in the
mean, which is at most the root mean square of dr' over that of r'.  Outputs
add half a unit of their type (2^-8 of a BF16 value, which has eight
significant bits, 2^-24 of an FP32 one)."""
import pytest
import torch

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def rms64(v, w, eps, off):
    return v / (v.pow(2).mean(1, keepdim=True) + eps).sqrt() * (off + w.double())


def want_64(r, w_pre, b, w_post, gate, scale, eps, off):
    z = torch.zeros_like(r.double()) if b is None else b.double()
    if w_post is not None:
        z = rms64(z, w_post, eps, off)
    if gate is not None:
        z = z * gate.double()
    t = scale * z
    rr = r.double() + t
    dr = 2.0 ** -16 * t.abs() + 2.0 ** -22 * r.double().abs()
    if w_pre is None:
        return rr, dr, None, None
    inv = 1 / (rr.pow(2).mean(1, keepdim=True) + eps).sqrt()
    n = rr * inv * (off + w_pre.double())
    rel = 2.0 ** -16 + dr.pow(2).mean(1, keepdim=True).sqrt() * inv
    return rr, dr, n, rel * n.abs() + (off + w_pre.double()).abs() * inv * dr


def check(got, want, bound, what):
    unit = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    bound = bound + unit * (want.abs() + bound) + 2.0 ** -126
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all(), what
    assert (err <= bound).all(), (what, float((err / bound).max()))


def inputs(M, H, res, gate, seed):
    g = torch.Generator().manual_seed(seed)
    r = (torch.randn(M, H, generator=g) * 2).to(res)
    b = (torch.randn(M, H, generator=g) * 0.3).to(BF16)
    w1 = (1 + 0.1 * torch.randn(H, generator=g)).to(BF16)
    w2 = (0.5 + 0.1 * torch.randn(H, generator=g)).to(BF16)
    shape = {"none": None, "channel": (H,), "token": (M, 1), "full": (M, H)}[gate]
    return r, b, w1, w2, None if shape is None else torch.randn(shape, generator=g).to(BF16)


def cu(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("M,H", [(1, 1), (1, 2560), (2, 7168), (3, 8), (5, 127), (7, 1283), (33, 264), (64, 4096),
                                 (2, 8192), (3, 8200), (2, 16384), (2, 16400), (1, 32768), (300, 512)])
@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_sandwich(M, H, res, gate):
    m = _m()
    r, b, pre, post, g = inputs(M, H, res, gate, M + H)
    rr, dr, n, dn = want_64(r, pre, b, post, g, 0.7, 1e-6, 0.0)
    got_r, got_n = m.block_norm(r.cuda(), pre.cuda(), b.cuda(), post_weight=post.cuda(), gate=cu(g), scale=0.7)
    assert got_r.dtype == res and got_n.dtype == BF16
    check(got_r, rr, dr, "residual")
    check(got_n, n, dn, "normed")


@pytest.mark.parametrize("M,H", [(333, 1), (333, 200), (333, 256), (334, 264), (1000, 505), (335, 506), (333, 512),
                                 (333, 513), (333, 2000), (333, 2042), (333, 4097), (333, 5005), (333, 5120),
                                 (310, 8191), (310, 8192), (2, 32761), (2, 32767)])
@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_many_rows(M, H, res, gate):
    """Enough rows for every arrangement of rows on warps and CTAs, packed and
    odd ones."""
    m = _m()
    r, b, pre, post, g = inputs(M, H, res, gate, M + H)
    if gate == "full" and H % 3 == 0:
        g = g.float()
    rr, dr, n, dn = want_64(r, pre, b, post, g, 0.7, 1e-6, 0.0)
    got_r, got_n = m.block_norm(r.cuda(), pre.cuda(), b.cuda(), post_weight=post.cuda(), gate=cu(g), scale=0.7)
    check(got_r, rr, dr, "residual")
    check(got_n, n, dn, "normed")


@pytest.mark.parametrize("M,H", [(5, 83), (400, 83), (400, 700), (400, 2100), (320, 4500)])
@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("at", [(0, 0, 0, 0), (3, 3, 3, 3), (4, 4, 4, 4), (7, 7, 7, 7), (5, 1, 5, 1), (1, 2, 3, 4)])
def test_rows_off_a_boundary(M, H, res, at):
    """Residual, block output, gate and output at columns `at` of wider
    buffers: off a 16-byte boundary alike, alike modulo four (enough for FP32
    rows beside BF16 ones, not for two BF16 ones), and each its own way. What
    lies around the rows stays."""
    m = _m()
    r, b, pre, post, g = inputs(M, H, res, "full", H)
    rr, dr, n, dn = want_64(r, pre, b, post, g, 0.7, 1e-6, 0.0)

    def wide(t, k):
        big = torch.full((M, H + 13), float("nan"), dtype=t.dtype, device="cuda")
        big[:, k:k + H] = t.cuda()
        return big[:, k:k + H]

    out = torch.full((M, H + 13), -7.0, dtype=res, device="cuda")
    got_r, got_n = m.block_norm(wide(r, at[0]), pre.cuda(), wide(b, at[1]), post_weight=post.cuda(),
                                gate=wide(g, at[2]), scale=0.7, residual_out=out[:, at[3]:at[3] + H])
    check(got_r, rr, dr, "residual")
    check(got_n, n, dn, "normed")
    assert (out[:, :at[3]] == -7).all() and (out[:, at[3] + H:] == -7).all()


@pytest.mark.parametrize("H", [256, 1000, 77])
def test_parts(H):
    """Each part left out; weights as FP32 differences from one; FP32 gates."""
    m = _m()
    M = 6
    r, b, pre, post, g = inputs(M, H, BF16, "full", H)
    R, B, PRE, POST = r.cuda(), b.cuda(), pre.cuda(), post.cuda()
    # the norm alone, which hands the residual back
    got_r, got_n = m.block_norm(R, PRE)
    assert got_r is R
    _, _, n, dn = want_64(r, pre, None, None, None, 1.0, 1e-6, 0.0)
    check(got_n, n, dn, "norm alone")
    # no norm after the block, no gate
    rr, dr, n, dn = want_64(r, pre, b, None, None, 1.0, 1e-6, 0.0)
    got_r, got_n = m.block_norm(R, PRE, B)
    check(got_r, rr, dr, "add")
    check(got_n, n, dn, "add norm")
    # no norm before the next block
    rr, dr, _, _ = want_64(r, None, b, post, None, 0.25, 1e-5, 0.0)
    got_r, got_n = m.block_norm(R, None, B, post_weight=POST, scale=0.25, eps=1e-5)
    assert got_n is None
    check(got_r, rr, dr, "post alone")
    # weights as differences from one, FP32 weights and gate
    w1, w2, g32 = (pre.float() - 1), (post.float() - 1), g.float()
    rr, dr, n, dn = want_64(r, w1, b, w2, g32, -1.5, 1e-6, 1.0)
    got_r, got_n = m.block_norm(R, w1.cuda(), B, post_weight=w2.cuda(), gate=g32.cuda(), scale=-1.5, weight_offset=1.0)
    check(got_r, rr, dr, "offset r")
    check(got_n, n, dn, "offset n")
    # in place
    R2 = R.clone()
    got_r, got_n2 = m.block_norm(R2, w1.cuda(), B, post_weight=w2.cuda(), gate=g32.cuda(), scale=-1.5,
                                 weight_offset=1.0, residual_out=R2)
    assert got_r is R2
    check(R2, rr, dr, "in place")
    assert torch.equal(got_n, got_n2)


@pytest.mark.parametrize("M,H", [(1, 16), (1, 4096), (3, 144), (9, 2560), (70, 7168), (2, 16384)])
@pytest.mark.parametrize("res", [BF16, F32])
def test_quantize_is_the_quantiser_of_normed(M, H, res):
    m = _m()
    r, b, pre, post, g = inputs(M, H, res, "token", 3)
    args = dict(post_weight=post.cuda(), gate=g.cuda(), scale=0.5)
    want_r, want_n = m.block_norm(r.cuda(), pre.cuda(), b.cuda(), **args)
    got_r, n, q, s = m.block_norm(r.cuda(), pre.cuda(), b.cuda(), quantize=True, **args)
    assert torch.equal(got_r, want_r) and torch.equal(n, want_n)
    wq, ws = m.fp8_quantize(n)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s, ws)


def test_strided_rows_and_zero_rows():
    m = _m()
    M, H = 11, 200
    r, b, pre, post, g = inputs(M, 2 * H, BF16, "full", 5)
    for off in (0, 8, 3):  # 16-byte aligned rows and unaligned ones
        sl = slice(off, off + H)
        rr, dr, n, dn = want_64(r[:, sl], pre[sl], b[:, sl], post[sl], g[:, sl], 1.0, 1e-6, 0.0)
        got_r, got_n = m.block_norm(r.cuda()[:, sl], pre.cuda()[sl], b.cuda()[:, sl], post_weight=post.cuda()[sl],
                                    gate=g.cuda()[:, sl])
        check(got_r, rr, dr, off)
        check(got_n, n, dn, off)
    zero = torch.zeros(4, H, dtype=BF16, device="cuda")
    got_r, got_n, q, s = m.block_norm(zero[:, :192], pre.cuda()[:192], zero[:, :192], post_weight=post.cuda()[:192],
                                      quantize=True)
    assert not got_r.any() and not got_n.any() and not q.view(torch.uint8).any() and (s == 1).all()
    assert m.block_norm(zero[:0], pre.cuda()[:H])[1].shape == (0, H)


def test_nonfinite_rows_stay_alone():
    m = _m()
    r, b, pre, post, _ = inputs(5, 512, BF16, "none", 6)
    b[1, 7], r[3, 9] = float("inf"), float("nan")
    got_r, got_n = m.block_norm(r.cuda(), pre.cuda(), b.cuda(), post_weight=post.cuda())
    for row in (0, 2, 4):
        assert torch.isfinite(got_r[row]).all() and torch.isfinite(got_n[row]).all()
    assert torch.isnan(got_n[1]).any() and torch.isnan(got_n[3]).all()


def test_large_values_do_not_overflow_the_output():
    """Rows whose sum of squares overflows FP32 (256 x 9e36 > 3.4e38) get a
    zero factor, as FP32 arithmetic does; large ones below that are normed."""
    m = _m()
    r = torch.full((2, 256), 1e15, dtype=BF16)
    r[1] = -3e18
    w = torch.ones(256, dtype=BF16)
    _, n = m.block_norm(r.cuda(), w.cuda())
    assert torch.allclose(n[0].float().cpu(), torch.ones(256), atol=2e-2)
    assert not n[1].any()


def test_refusals():
    m = _m()
    r, b, pre, post, g = (cu(t) for t in inputs(4, 64, BF16, "full", 1))
    for bad in (dict(block_out=b.float()), dict(block_out=b, gate=g.half())):
        with pytest.raises(TypeError):
            m.block_norm(r, pre, **bad)
    with pytest.raises(TypeError):
        m.block_norm(r.half(), pre)
    with pytest.raises(TypeError):
        m.block_norm(r, pre, b, post_weight=post.float())  # both weights have one type
    with pytest.raises(TypeError):
        m.block_norm(r, pre, b, residual_out=torch.empty(4, 64, device="cuda"))
    for bad in (dict(block_out=b[:, :32]), dict(post_weight=post), dict(gate=g), dict(block_out=b, gate=g[:, :3]),
                dict(block_out=b, gate=g.t().contiguous().t()), dict(block_out=b.cpu())):
        with pytest.raises(ValueError):
            m.block_norm(r, pre, **bad)
    with pytest.raises(ValueError):
        m.block_norm(r, pre[:32])
    with pytest.raises(ValueError):
        m.block_norm(r)
    with pytest.raises(ValueError):
        m.block_norm(r, None, b, quantize=True)
    with pytest.raises(ValueError):
        m.block_norm(r.cpu(), pre)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf")), dict(weight_offset=float("nan"))):
        with pytest.raises(m.MoeFp4Error):
            m.block_norm(r, pre, b, **bad)
    with pytest.raises(m.MoeFp4Error):
        m.block_norm(r[:, :24], pre[:24], quantize=True)  # H % 16
    with pytest.raises(m.MoeFp4Error):
        m.block_norm(r[:, 1:17], pre[1:17], quantize=True)  # unaligned rows
