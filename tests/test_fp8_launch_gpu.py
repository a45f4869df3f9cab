"""The FP8 products' launches beside other work of the program."""
import os
import subprocess
import sys

import pytest
import torch

from tests.gpu_util import ensure_built
from tests.test_fp8_gpu import blocks, rand_fp8, rand_scale

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

AFTER_A_REFUSED_CALL = """
import torch
import fp4_weight_moe_gb300 as m
x = torch.randn(64, 512, device="cuda").to(torch.bfloat16)
w, ws = torch.randn(256, 512, device="cuda").to(torch.float8_e4m3fn), torch.rand(2, 4, device="cuda")
want = m.fp8_linear(x, w, ws)
graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(stream):
    graph.capture_begin()
    try:
        m.fp8_status()
        raise SystemExit("the status was read during a capture")
    except m.MoeFp4Error:
        pass
    try:
        graph.capture_end()
    except RuntimeError:
        pass
torch.cuda.synchronize()
for _ in range(2):
    assert torch.equal(m.fp8_linear(x, w, ws), want)
print("fine")
"""


def test_linear_after_a_refused_call():
    """A call that the runtime refused (a status read, which synchronises,
    during a capture) was reported by its own status; the next fp8_linear
    neither reports it again nor stops between its two launches. (In a process
    of its own: the capture is spoilt.)"""
    ensure_built()
    r = subprocess.run([sys.executable, "-c", AFTER_A_REFUSED_CALL], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout[-2000:] + r.stderr[-2000:]


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
