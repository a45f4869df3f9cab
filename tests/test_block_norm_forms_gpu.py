"""block_norm's FP8 form where many rows take a warp or few chunks a thread
each, and where a row fills the widest CTA."""
import pytest
import torch

from tests.gpu_util import ensure_built
from tests.test_block_norm_gpu import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,H", [(333, 16), (333, 272), (2600, 256), (333, 512), (2600, 496), (333, 528), (333, 1040),
                                 (333, 2048), (333, 2064), (2600, 4096), (333, 4112), (333, 5120), (2600, 7168),
                                 (333, 8192), (333, 8208), (3, 16400), (2, 32768)])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["token", "full"])
def test_quantize_is_the_quantiser_of_normed(M, H, res, gate):
    ensure_built()
    import fp4_weight_moe_gb300 as m
    r, b, pre, post, g = inputs(M, H, res, gate, H)
    args = dict(post_weight=post.cuda(), gate=g.cuda(), scale=0.5)
    want_r, want_n = m.block_norm(r.cuda(), pre.cuda(), b.cuda(), **args)
    got_r, n, q, s = m.block_norm(r.cuda(), pre.cuda(), b.cuda(), quantize=True, **args)
    assert torch.equal(got_r, want_r) and torch.equal(n, want_n)
    wq, ws = m.fp8_quantize(n)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s, ws)
