"""The forms of the FP8 quantiser and product that prompts run in: many tiles
with K past one chunk of scales, fp8_linear's early loads and padded scales on
them, and the quantiser of many rows in every activation.

Bounds of a product as in tests/test_fp8_gpu.py."""
import pytest
import torch

from tests.gpu_util import ensure_built
from tests.test_fp8_gpu import blocks, check, product_64, quantised_32, rand_fp8, rand_scale

pytestmark = pytest.mark.gpu


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


@pytest.mark.parametrize("M,K,N", [(1300, 7168, 1100), (1300, 2064, 1111), (2001, 7168, 1500), (2001, 2176, 1500),
                                   (4100, 2176, 2816), (2603, 4112, 2101)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_many_tiles_long_k(M, K, N, out):
    """Seventeen and more K blocks a tile, 128 and 256 columns wide, several
    tiles a CTA; both layouts of the activation scales, the same bits again."""
    m = _m()
    xq, wq = rand_fp8(M, K, 1).cuda(), rand_fp8(N, K, 2).cuda()
    xs, ws = rand_scale(M, blocks(K), 3).cuda(), rand_scale(blocks(N), blocks(K), 4).cuda()
    want, mag = (t.cpu() for t in product_64(xq, xs, wq, ws))
    got = m.fp8_matmul(xq, xs, wq, ws, out_dtype=out)
    check(got, want, mag, K, out)
    turned = xs.t().contiguous().t()
    for _ in range(5):
        assert torch.equal(m.fp8_matmul(xq, turned, wq, ws, out_dtype=out), got)
    assert m.fp8_status() == 0


@pytest.mark.parametrize("M,K,N", [(2601, 384, 2048), (2003, 272, 2101), (1301, 7168, 1100), (2602, 2176, 1500),
                                   (46, 4096, 640)])
def test_linear_is_quantize_then_matmul_many_tiles(M, K, N):
    """The same bits as the two calls where tokens are no multiple of four, on
    one workspace, with weights that the stream wrote just before."""
    m = _m()
    g = torch.Generator(device="cuda").manual_seed(M)
    xs = [torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    ws = [rand_fp8(N, K, i).cuda() for i in range(3)]
    scales = [rand_scale(blocks(N), blocks(K), 10 + i).cuda() for i in range(3)]
    want = [m.fp8_matmul(*m.fp8_quantize(x), w, s, out_dtype=torch.float32) for x, w, s in zip(xs, ws, scales)]
    work = m.alloc_fp8_workspace(M, K)
    work.fill_(0xFF)  # (NaN in the rows past the last)
    w = torch.empty_like(ws[0])
    s = torch.empty_like(scales[0])
    got = []
    for i in (0, 1, 2, 0, 2, 1):
        w.view(torch.uint8).copy_(ws[i].view(torch.uint8))
        s.copy_(scales[i])
        got.append((i, m.fp8_linear(xs[i], w, s, out_dtype=torch.float32, workspace=work)))
    for i, y in got:
        assert torch.equal(y, want[i])
    assert m.fp8_status() == 0


@pytest.mark.parametrize("M,K", [(700, 7168), (1000, 2576), (1500, 1040), (2500, 512)])
def test_quantize_many_rows(M, K):
    m = _m()
    g = torch.Generator().manual_seed(K)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    x[:, ::7] *= 30
    x[1, K - 16:] = 0
    x[2] = 1e-38
    q, s = m.fp8_quantize(x.cuda())
    want_q, want_s = quantised_32(x.float())
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(q.cpu().view(torch.uint8), want_q)


@pytest.mark.parametrize("M,K", [(700, 7168), (1000, 2576), (1500, 1040), (2500, 512)])
@pytest.mark.parametrize("kind", ["silu", "gelu", "oai"])
def test_quantize_gated_many_rows(M, K, kind):
    """Half an E4M3 step of the value and 2^-12 of the block's largest, and
    the bits of a few rows at a time."""
    m = _m()
    g = torch.Generator().manual_seed(K + M)
    x = (torch.randn(M, 2 * K, generator=g) * 2).to(torch.bfloat16)
    gate, up = x[:, :K].double(), x[:, K:].double()
    if kind == "silu":
        v, args = gate * torch.sigmoid(gate) * up, dict(act=m.ACT_SILU)
    elif kind == "gelu":
        v = 0.5 * gate * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (gate + 0.044715 * gate ** 3))) * up
        args = dict(act=m.ACT_GELU_TANH)
    else:
        gc = gate.clamp(max=3.0)
        v = (up.clamp(-3.0, 3.0) + 1.0) * gc * torch.sigmoid(1.702 * gc)
        args = dict(act=m.ACT_SWIGLUOAI, alpha=1.702, beta=1.0, limit=3.0)
    x = x.cuda()
    q, s = m.fp8_quantize(x, **args)
    s64 = s.cpu().double().repeat_interleave(128, 1)[:, :K]
    bound = v.abs() / 16 + s64 * 2.0 ** -10 + 448 * s64 * 2.0 ** -12
    assert ((q.cpu().double() * s64 - v).abs() <= bound).all()
    for at in range(0, M, 100):
        few_q, few_s = m.fp8_quantize(x[at:at + 100], **args)
        assert torch.equal(few_q.view(torch.uint8), q[at:at + 100].view(torch.uint8))
        assert torch.equal(few_s, s[at:at + 100])
