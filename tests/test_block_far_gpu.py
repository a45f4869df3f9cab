"""The operators around the layer on rows whose offsets pass 32 bits: the
same bits as on compact copies of the rows."""
import pytest
import torch

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
M, ROW = 2100, (1 << 20) + 32  # 2.2e9 elements


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


@pytest.fixture
def far():
    """bf16 rows far apart; what lies between them is never initialised."""
    return torch.empty(M, ROW, dtype=torch.bfloat16, device="cuda")


def rows(far, at, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(M, cols, generator=g, device="cuda").to(torch.bfloat16)
    far[:, at:at + cols] = v
    return far[:, at:at + cols], v


def test_norm(far):
    m = _m()
    H = 512
    R, r = rows(far, 8, H, 1)
    B, b = rows(far, 1024, H, 2)
    G, g = rows(far, 2048, H, 3)
    out = far[:, 4096:4096 + H]
    w = torch.rand(H, device="cuda").to(torch.bfloat16)
    want_r, want_n = m.block_norm(r, w, b, post_weight=w, gate=g)
    got_r, got_n = m.block_norm(R, w, B, post_weight=w, gate=G, residual_out=out)
    assert torch.equal(got_r, want_r) and torch.equal(got_n, want_n)
    # rows off a 16-byte boundary, alike
    R, r = rows(far, 3, 501, 4)
    B, b = rows(far, 1027, 501, 5)
    got_r, got_n = m.block_norm(R, w[:501].contiguous(), B, residual_out=far[:, 4099:4099 + 501])
    torch.testing.assert_close(got_r, (r.float() + b.float()).to(torch.bfloat16), rtol=2.0 ** -7, atol=1e-6)
    assert torch.isfinite(got_n).all()


def test_product_and_quantiser(far):
    m = _m()
    K, N = 256, 400
    X, x = rows(far, 16, K, 1)
    W = torch.randn(N, K, device="cuda").to(torch.float8_e4m3fn)
    ws = torch.rand(4, 2, device="cuda")
    want_q, want_s = m.fp8_quantize(x)
    q, s = m.fp8_quantize(X)
    assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
    A, add = rows(far, 8192, N, 2)
    want = m.fp8_matmul(q, s, W, ws, addend=add)
    for at in (4096, 4099):  # vector stores, single ones
        got = m.fp8_matmul(q, s, W, ws, addend=A, out=far[:, at:at + N])
        assert torch.equal(got, want)
    # quantised rows far apart (bytes of the same buffer)
    Q = far.view(torch.uint8)[:, 20000:20000 + K]
    Q.copy_(q.view(torch.uint8))
    assert torch.equal(m.fp8_matmul(Q.view(torch.float8_e4m3fn), s, W, ws, addend=add), want)
    assert torch.equal(m.fp8_linear(X, W, ws, addend=A), want)
    assert m.fp8_status() == 0


def test_router(far):
    m = _m()
    L, logits = rows(far, 40, 200, 1)
    got, want = m.route_topk(L, 6), m.route_topk(logits, 6)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
