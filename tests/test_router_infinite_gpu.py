"""Infinite logits in the router's choice."""
import pytest
import torch

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("E", [40, 300, 1500])
@pytest.mark.parametrize("renorm", [True, False])
def test_infinite_logits(E, renorm):
    """An expert with a logit of +inf comes first; the softmax of its row is
    undefined, and all weights chosen there are NaN (as torch.softmax gives
    them), never an ordinary value. The sigmoid gives such an expert a score
    of one."""
    ensure_built()
    import fp4_weight_moe_gb300 as m
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(4, E, generator=g)
    logits[1, 7] = INF
    logits[2, 9], logits[2, 30] = INF, INF
    logits[3, 3:] = -INF
    logits[3, 1] = INF
    x = logits.cuda()
    ids, w = (t.cpu() for t in m.route_topk(x, 8, renormalize=renorm))
    soft = torch.softmax(logits.double(), 1)
    assert soft[1:].isnan().any(1).all()
    assert torch.equal(ids[0].long(), logits[0].topk(8).indices) and torch.isfinite(w[0]).all()
    assert ids[1, 0] == 7 and ids[2, :2].tolist() == [9, 30] and w[1].isnan().all() and w[2].isnan().all()
    assert ids[3, 0] == 1 and (ids[3, 3:] == -1).all() and w[3, :3].isnan().all() and not w[3, 3:].any()
    ids, w = (t.cpu() for t in m.route_topk(x, 8, score=m.SCORE_SIGMOID, renormalize=False))
    assert ids[1, 0] == 7 and w[1, 0] == 1 and ids[2, :2].tolist() == [9, 30] and (w[2, :2] == 1).all()
    assert torch.isfinite(w).all()
