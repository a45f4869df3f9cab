"""The FP8 products with a scale per block of 128 and their activation
quantiser, against the definition in 64 bits.

Bounds.  A product of two E4M3 values is exact in FP32, so an element's error
comes from FP32 sums alone: 128 terms in a block, one scaled addition per
block, one product of two scales; each operation is off by at most 2^-23 of
the sum of magnitudes so far, whatever its order.  With A = sum_b sx sw
sum_k |x w|, |error| <= (128 + blocks + 4) 2^-23 A, and the output adds half a
unit of its type (2^-8 |y| for BF16, which has eight significant bits) after
the addend."""
import numpy as np
import pytest
import torch

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def blocks(n):
    return (n + 127) // 128


def rand_fp8(rows, cols, seed, big=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g) * (100.0 if big else 3.0)
    return v.clamp(-448, 448).to(torch.float8_e4m3fn)


def rand_scale(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.exp(torch.randn(rows, cols, generator=g)) * 1e-2


def product_64(xq, xs, wq, ws):
    """(product, sum of magnitudes) in 64 bits."""
    K, N = xq.shape[1], wq.shape[0]
    x = xq.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    w = wq.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x @ w.t(), x.abs() @ w.abs().t()


def check(got, want, mag, K, out_dtype, add=None):
    if add is not None:
        want = want + add.double()
        mag = mag + add.double().abs()
    bound = (128 + blocks(K) + 4) * 2.0 ** -23 * mag
    if out_dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound) + 2.0 ** -134
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= bound).all(), float((err / bound.clamp(min=1e-300)).max())


SIZES = [(1, 128, 128), (1, 16, 1), (2, 7168, 256), (3, 272, 130), (8, 2560, 640), (9, 400, 129), (16, 2048, 513),
         (17, 144, 1000), (33, 1024, 384), (64, 4096, 264), (65, 256, 72), (100, 2576, 136), (128, 128, 128),
         (129, 2064, 257), (200, 512, 1032), (256, 1280, 512), (300, 640, 2000), (513, 384, 700), (1025, 272, 1100),
         (2500, 896, 2100)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_matmul(M, K, N, out):
    m = _m()
    xq, wq = rand_fp8(M, K, 1, big=True), rand_fp8(N, K, 2)
    xs, ws = rand_scale(M, blocks(K), 3), rand_scale(blocks(N), blocks(K), 4)
    want, mag = product_64(xq, xs, wq, ws)
    got = m.fp8_matmul(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out_dtype=out)
    assert got.dtype == out
    check(got, want, mag, K, out)
    # block-major scales (what the quantiser writes): the same bits
    again = m.fp8_matmul(xq.cuda(), xs.t().contiguous().cuda().t(), wq.cuda(), ws.cuda(), out_dtype=out)
    assert torch.equal(got, again)
    assert m.fp8_status() == 0


@pytest.mark.parametrize("M,K,N,at", [(2000, 256, 2101, 0), (2001, 144, 2102, 0), (2002, 272, 2104, 1),
                                      (2003, 128, 2112, 8), (1999, 256, 2100, 3), (4100, 400, 2816, 0)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_add", [False, True])
def test_many_tiles_any_row_start(M, K, N, at, out, with_add):
    """More tiles than SMs, rows of the output that start at any value: the
    stores of whole sectors, of vectors, of pairs and of single values."""
    m = _m()
    xq, wq = rand_fp8(M, K, 1), rand_fp8(N, K, 2)
    xs, ws = rand_scale(M, blocks(K), 3), rand_scale(blocks(N), blocks(K), 4)
    add = torch.randn(M, N, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16) if with_add else None
    want, mag = product_64(xq, xs, wq, ws)
    buf = torch.full((M, N + at), -7.0, dtype=out, device="cuda")
    s = xs.t().contiguous().cuda().t()
    m.fp8_matmul(xq.cuda(), s, wq.cuda(), ws.cuda(), out=buf[:, at:], addend=None if add is None else add.cuda())
    check(buf[:, at:], want, mag, K, out, add)
    assert (buf[:, :at] == -7).all()


@pytest.mark.parametrize("M", [1, 8, 16, 24, 32, 64, 128])
def test_long_k_per_cta(M):
    """Sixteen K blocks and more to a CTA, so that every form's ring of stages
    goes round several times, many calls in a row; the self-quantising form
    (up to eight tokens) gives the bits of the two calls."""
    m = _m()
    K, N = 16384, 384
    wq, ws = rand_fp8(N, K, 2), rand_scale(blocks(N), blocks(K), 4)
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    q, s = m.fp8_quantize(x)
    want, mag = product_64(q.cpu(), s.cpu(), wq, ws)
    W, WS = wq.cuda(), ws.cuda()
    first = m.fp8_matmul(q, s, W, WS, out_dtype=torch.float32)
    check(first, want, mag, K, torch.float32)
    for _ in range(20):
        assert torch.equal(m.fp8_matmul(q, s, W, WS, out_dtype=torch.float32), first)
        assert torch.equal(m.fp8_linear(x, W, WS, out_dtype=torch.float32), first)
    assert m.fp8_status() == 0


@pytest.mark.parametrize("M,K,N", [(24, 7168, 7168), (17, 5120, 5000), (30, 2048, 20000)])
def test_many_tiles_few_tokens(M, K, N):
    m = _m()
    xq, wq = rand_fp8(M, K, 1), rand_fp8(N, K, 2)
    xs, ws = rand_scale(M, blocks(K), 3), rand_scale(blocks(N), blocks(K), 4)
    want, mag = product_64(xq, xs, wq, ws)
    args = xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda()
    first = m.fp8_matmul(*args)
    check(first, want, mag, K, torch.bfloat16)
    for _ in range(20):
        assert torch.equal(m.fp8_matmul(*args), first)
    assert m.fp8_status() == 0


@pytest.mark.parametrize("M,K,N", [(1, 7168, 512), (5, 272, 129), (40, 512, 384), (300, 640, 500)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_matmul_addend_and_strides(M, K, N, out):
    """Rows with strides and offsets of their own on every operand; the addend
    joins before the rounding; the padding of out stays untouched."""
    m = _m()
    g = torch.Generator().manual_seed(9)
    xq, wq = rand_fp8(M, K, 5), rand_fp8(N, K, 6)
    xs, ws = rand_scale(M, blocks(K), 7), rand_scale(blocks(N), blocks(K), 8)
    add = torch.randn(M, N, generator=g).to(torch.bfloat16)
    want, mag = product_64(xq, xs, wq, ws)

    def wide(t, before, after):
        big = torch.zeros(t.shape[0], before + t.shape[1] + after, dtype=torch.uint8).view(torch.uint8) \
            if t.dtype == torch.float8_e4m3fn else torch.zeros(t.shape[0], before + t.shape[1] + after, dtype=t.dtype)
        src = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
        big[:, before:before + t.shape[1]] = src
        big = big.cuda()
        v = big[:, before:before + t.shape[1]]
        return v.view(torch.float8_e4m3fn) if t.dtype == torch.float8_e4m3fn else v

    buf = torch.full((M, N + 11), -7.0, dtype=out, device="cuda")
    got = m.fp8_matmul(wide(xq, 16, 32), wide(xs, 3, 2), wide(wq, 32, 16), wide(ws, 1, 4), out=buf[:, 3:3 + N],
                       addend=wide(add, 5, 2))
    assert got.data_ptr() == buf[:, 3:].data_ptr()
    check(got, want, mag, K, out, add)
    assert (buf[:, :3] == -7).all() and (buf[:, 3 + N:] == -7).all()


def test_matmul_in_place_addend_and_zero_rows():
    m = _m()
    M, K, N = 37, 384, 200
    xq, wq = rand_fp8(M, K, 1), rand_fp8(N, K, 2)
    xq.view(torch.uint8)[5] = 0
    xs, ws = rand_scale(M, 3, 3), rand_scale(2, 3, 4)
    add = torch.randn(M, N).to(torch.bfloat16)
    want, mag = product_64(xq, xs, wq, ws)
    buf = add.cuda()
    m.fp8_matmul(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out=buf, addend=buf)
    check(buf, want, mag, K, torch.bfloat16, add)
    assert torch.equal(buf[5].cpu(), add[5])
    empty = m.fp8_matmul(xq.cuda()[:0], xs.cuda()[:0], wq.cuda(), ws.cuda())
    assert empty.shape == (0, N)


def test_matmul_nan_stays_in_its_row():
    m = _m()
    for M in (3, 70, 300):
        K, N = 512, 300
        xq, wq = rand_fp8(M, K, 1), rand_fp8(N, K, 2)
        xq.view(torch.uint8)[1, 200] = 0x7F  # NaN
        xs, ws = rand_scale(M, 4, 3), rand_scale(3, 4, 4)
        y = m.fp8_matmul(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda()).cpu()
        assert torch.isnan(y[1]).all()
        assert torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def quantised_32(x):
    """The quantiser's definition on CPU float32 values, step by step."""
    M, K = x.shape
    pad = torch.nn.functional.pad(x, (0, blocks(K) * 128 - K)).view(M, -1, 128)
    s = pad.abs().amax(2, keepdim=True)
    s = s / torch.full_like(s, 448.0)
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (pad / s).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(M, -1)[:, :K], s[:, :, 0]


@pytest.mark.parametrize("M,K", [(1, 16), (1, 7168), (3, 128), (7, 144), (33, 2576), (1000, 256)])
def test_quantize_bits(M, K):
    m = _m()
    g = torch.Generator().manual_seed(M * K)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    x[:, ::7] *= 30
    x[0, : min(K, 128)] = 0          # an all-zero block
    if M > 2:
        x[1] = 1e-38                 # tiny values
        x[2, 0] = 3e38               # a huge one
    q, s = m.fp8_quantize(x.cuda())
    want_q, want_s = quantised_32(x.float())
    assert q.dtype == torch.float8_e4m3fn and s.shape == (M, blocks(K))
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(q.cpu().view(torch.uint8), want_q)


def test_quantize_rows_with_a_stride():
    m = _m()
    x = torch.randn(9, 512).to(torch.bfloat16).cuda()
    q, s = m.fp8_quantize(x[:, 64:64 + 272])
    want_q, want_s = quantised_32(x[:, 64:64 + 272].float().cpu())
    assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu().view(torch.uint8), want_q)


@pytest.mark.parametrize("M,K", [(1, 2048), (5, 272), (64, 384)])
@pytest.mark.parametrize("kind", ["silu", "gelu", "oai"])
def test_quantize_gated(M, K, kind):
    """Dequantised values against act(gate) * up in 64 bits: half an E4M3
    step of the value (1/16 of it, or 2^-10 scales below the normals), and
    2^-12 of the block's largest for the FP32 activation and scale."""
    m = _m()
    g = torch.Generator().manual_seed(K + M)
    x = (torch.randn(M, 2 * K, generator=g) * 2).to(torch.bfloat16)
    gate, up = x[:, :K].double(), x[:, K:].double()
    if kind == "silu":
        v = gate * torch.sigmoid(gate) * up
        q, s = m.fp8_quantize(x.cuda(), act=m.ACT_SILU)
    elif kind == "gelu":
        v = 0.5 * gate * (1 + torch.tanh((2 / np.pi) ** 0.5 * (gate + 0.044715 * gate ** 3))) * up
        q, s = m.fp8_quantize(x.cuda(), act=m.ACT_GELU_TANH)
    else:
        gc, uc = gate.clamp(max=3.0), up.clamp(-3.0, 3.0)
        v = (uc + 1.0) * gc * torch.sigmoid(1.702 * gc)
        q, s = m.fp8_quantize(x.cuda(), act=m.ACT_SWIGLUOAI, alpha=1.702, beta=1.0, limit=3.0)
    s64 = s.cpu().double().repeat_interleave(128, 1)[:, :K]
    got = q.cpu().double() * s64
    bound = v.abs() / 16 + s64 * 2.0 ** -10 + 448 * s64 * 2.0 ** -12
    assert ((got - v).abs() <= bound).all()


@pytest.mark.parametrize("rows", [1024, 65536])
def test_quantize_silu_bits(rows):
    """SiLU(g) * 1 of every BF16 g, alone in its row, through its scale: each
    step an IEEE operation on the GPU's own expf. (1024 rows at a time and all
    at once take the two forms of the kernel.)"""
    m = _m()
    g = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    x = torch.zeros(65536, 32, dtype=torch.bfloat16, device="cuda")
    x[:, :16] = 2.0 ** -10
    x[:, 5], x[:, 21] = g, 1.0
    got = torch.cat([m.fp8_quantize(c, act=m.ACT_SILU)[1] for c in x.split(rows)])[:, 0]
    f = g.float()
    v = (f / (1.0 + torch.exp(-f))).abs()
    want = torch.where(v.isnan(), torch.zeros_like(v), v)  # (NaNs are passed over)
    want = want / torch.full_like(want, 448.0)
    want = torch.where(want == 0, torch.ones_like(want), want)
    assert torch.equal(got, want), (got != want).sum()


def test_quantize_every_scale_significand():
    """v / s with the scale of every BF16 maximum's significand, small and
    large, and v at every 128th of the maximum."""
    m = _m()
    top = (torch.arange(128, dtype=torch.int32) + 128).float()  # every BF16 significand
    lead = torch.tensor([2.0 ** e for e in (-58, -40, 0, 30, 50)])
    amax = (top[:, None] * lead[None]).reshape(-1)
    ratios = torch.arange(1, 129, dtype=torch.float32) / 128
    x = torch.zeros(amax.numel(), 144)
    x[:, :128] = amax[:, None] * ratios[None]
    x = x.to(torch.bfloat16)
    x[:, 127] = amax.to(torch.bfloat16)
    want_q, want_s = quantised_32(x.float())
    for rows in (x, x.repeat(8, 1)):  # (the two forms of the kernel)
        q, s = m.fp8_quantize(rows.cuda())
        for c in range(0, rows.shape[0], x.shape[0]):
            assert torch.equal(s[c:c + x.shape[0]].cpu(), want_s)
            assert torch.equal(q[c:c + x.shape[0]].cpu().view(torch.uint8), want_q)


@pytest.mark.parametrize("M,K,N", [(1, 2560, 300), (4, 272, 640), (16, 7168, 128), (17, 512, 1000), (150, 640, 257)])
def test_linear_is_quantize_then_matmul(M, K, N):
    """The same bits as the two calls, with and without a workspace."""
    m = _m()
    g = torch.Generator().manual_seed(11)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    wq, ws = rand_fp8(N, K, 2).cuda(), rand_scale(blocks(N), blocks(K), 4).cuda()
    add = torch.randn(M, N, generator=g).to(torch.bfloat16).cuda()
    q, s = m.fp8_quantize(x)
    want = m.fp8_matmul(q, s, wq, ws, addend=add)
    w = m.alloc_fp8_workspace(M + 3, K)
    assert torch.equal(m.fp8_linear(x, wq, ws, addend=add), want)
    assert torch.equal(m.fp8_linear(x, wq, ws, addend=add, workspace=w), want)
    p, mag = product_64(q.cpu(), s.cpu(), wq.cpu(), ws.cpu())
    check(want, p, mag, K, torch.bfloat16, add.cpu())
    with pytest.raises(m.MoeFp4Error) as e:
        m.fp8_linear(x, wq, ws, workspace=w[:256])
    assert e.value.status == m._capi.MOE_FP4_EWORKSPACE


def test_on_another_stream_and_in_a_graph():
    m = _m()
    M, K, N = 6, 1024, 512
    x = torch.randn(M, K).to(torch.bfloat16).cuda()
    wq, ws = rand_fp8(N, K, 2).cuda(), rand_scale(4, 8, 4).cuda()
    want = m.fp8_linear(x, wq, ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = m.fp8_linear(x, wq, ws, stream=st)
    st.synchronize()
    assert torch.equal(y, want)
    w, out = m.alloc_fp8_workspace(M, K), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.fp8_linear(x, wq, ws, out=out, workspace=w)
    x.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, m.fp8_linear(x, wq, ws))


def test_refusals():
    m = _m()
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w, ws = torch.zeros(64, 256, device="cuda").to(torch.float8_e4m3fn), torch.ones(1, 2, device="cuda")
    q, s = m.fp8_quantize(x)
    with pytest.raises(TypeError):
        m.fp8_linear(x.float(), w, ws)
    with pytest.raises(TypeError):
        m.fp8_linear(x, w.view(torch.uint8), ws)
    with pytest.raises(TypeError):
        m.fp8_linear(x, w, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        m.fp8_linear(x, w, torch.ones(1, 3, device="cuda"))
    with pytest.raises(ValueError):
        m.fp8_linear(x, w[:, :128], ws[:, :1])
    with pytest.raises(ValueError):
        m.fp8_matmul(q, s[:, :1], w, ws)
    with pytest.raises(ValueError):
        m.fp8_linear(x.cpu(), w, ws)
    with pytest.raises(ValueError):
        m.fp8_linear(x, w.cpu(), ws)
    with pytest.raises(ValueError):
        m.fp8_linear(x, w, ws, addend=torch.zeros(4, 63, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        m.fp8_quantize(torch.zeros(4, 31, dtype=torch.bfloat16, device="cuda"), act=m.ACT_SILU)
    for bad in (lambda: m.fp8_quantize(x[:, :24]), lambda: m.fp8_quantize(x[:, 1:17]),
                lambda: m.fp8_quantize(x, act=m.ACT_RELU2), lambda: m.fp8_linear(x[:, 4:20], w[:, :16], ws[:, :1])):
        with pytest.raises(m.MoeFp4Error):
            bad()
