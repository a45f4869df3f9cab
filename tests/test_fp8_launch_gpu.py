"""The FP8 products' launches beside other work of the program."""
import pytest
import torch

from tests.gpu_util import ensure_built
from tests.test_fp8_gpu import blocks, rand_fp8, rand_scale

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [3, 40, 700])
def test_each_call_reads_what_the_one_before_wrote(M):
    """Norm, quantiser and products launch as dependents of the launch before
    them: inputs rewritten by that launch, over and over in the same buffers,
    are read after it."""
    ensure_built()
    import fp4_weight_moe_gb300 as m
    H, I = 1024, 384
    g = torch.Generator(device="cuda").manual_seed(M)
    steps = [torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(12)]
    w_pre = torch.rand(H, generator=g, device="cuda").to(torch.bfloat16)
    up, up_s = rand_fp8(2 * I, H, 1).cuda(), rand_scale(blocks(2 * I), blocks(H), 2).cuda()
    down, down_s = rand_fp8(H, I, 3).cuda(), rand_scale(blocks(H), blocks(I), 4).cuda()

    def run(wait):
        stream, gu, out = steps[0].clone(), torch.zeros(M, 2 * I, dtype=torch.bfloat16, device="cuda"), []
        y = torch.zeros_like(stream)
        for step in steps:
            y.add_(step)
            wait()
            _, n = m.block_norm(stream, w_pre, y, residual_out=stream)
            wait()
            m.fp8_linear(n, up, up_s, out=gu)
            wait()
            q, s = m.fp8_quantize(gu, act=m.ACT_SILU)
            wait()
            m.fp8_matmul(q, s, down, down_s, out=y, addend=n)
            wait()
            out += [stream.clone(), q.view(torch.uint8).clone(), y.clone()]
        return out

    want = run(torch.cuda.synchronize)
    for _ in range(10):
        got = run(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
