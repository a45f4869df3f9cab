"""The same sizes with outputs at different alignments: each within the bound
of tests/test_fp8_gpu.py, and each the same bits every time."""
import pytest
import torch

from tests.gpu_util import ensure_built
from tests.test_fp8_gpu import blocks, check, product_64, rand_fp8, rand_scale

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [(300, 1024, 1024), (64, 512, 640), (3, 2048, 512), (700, 2176, 2112)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_each_alignment_has_its_bits(M, K, N, out):
    ensure_built()
    import fp4_weight_moe_gb300 as m
    xq, wq = rand_fp8(M, K, 1), rand_fp8(N, K, 2)
    xs, ws = rand_scale(M, blocks(K), 3), rand_scale(blocks(N), blocks(K), 4)
    want, mag = product_64(xq, xs, wq, ws)
    args = xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda()
    for at in (0, 1, 2, 4, 8):
        buf = torch.zeros(M, N + 16, dtype=out, device="cuda")
        first = m.fp8_matmul(*args, out=buf[:, at:at + N]).clone()
        check(first, want, mag, K, out)
        for _ in range(3):
            assert torch.equal(m.fp8_matmul(*args, out=buf[:, at:at + N]), first)
