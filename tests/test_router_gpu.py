"""The router's choice against its definition: ids exactly (the order is by
FP32 scores, ties to the lowest index), weights against 64 bits.

Bound of a weight: expf and the sigmoid are off by less than 2^-21 of
themselves, the sums of at most 65536 positive terms by 2^-18, the division
by 2^-24."""
import pytest
import torch

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def want(logits, k, sigmoid, bias, renorm, scale):
    """ids by the definition in FP32 on the CPU (scores from the GPU's expf
    where it matters: the caller passes scores that have no near ties), and
    weights in 64 bits."""
    l64 = logits.double()
    fine = logits.float() > float("-inf")
    order = l64 if not sigmoid else torch.sigmoid(l64) + (0 if bias is None else bias.double())
    order = torch.where(fine, order, torch.full_like(order, float("-inf")))
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    taken = torch.gather(fine, 1, ids)
    if sigmoid:
        s = torch.sigmoid(l64)
    else:
        top = torch.where(fine, l64, torch.full_like(l64, float("-inf"))).amax(1, keepdim=True)
        s = torch.where(fine, torch.exp(l64 - torch.where(top > float("-inf"), top, torch.zeros_like(top))),
                        torch.zeros_like(l64))
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    w = torch.where(taken, torch.gather(torch.nan_to_num(s), 1, ids), torch.zeros_like(ids, dtype=torch.float64))
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return torch.where(taken, ids, torch.full_like(ids, -1)).int(), w * scale


def check(m, logits, k, sigmoid=False, bias=None, renorm=True, scale=1.0):
    ids, w = m.route_topk(logits.cuda(), k, score=m.SCORE_SIGMOID if sigmoid else m.SCORE_SOFTMAX,
                          bias=None if bias is None else bias.cuda(), renormalize=renorm, scale=scale)
    want_ids, want_w = want(logits, k, sigmoid, bias, renorm, scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32 and ids.shape == w.shape == (logits.shape[0], k)
    assert torch.equal(ids.cpu(), want_ids)
    err = (w.cpu().double() - want_w).abs()
    assert (err <= 2.0 ** -16 * want_w.abs() + 1e-37).all()
    return ids, w


SIZES = [(1, 1, 1), (1, 8, 2), (4, 288, 10), (3, 33, 16), (7, 16, 16), (5, 31, 7), (64, 512, 10), (9, 130, 8),
         (2, 1000, 16), (3, 1024, 4), (2, 1025, 9), (2, 4096, 8), (1, 65536, 16), (1000, 128, 8), (37, 64, 6),
         (2049, 256, 8)]


@pytest.mark.parametrize("M,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_softmax(M, E, k, dtype, renorm):
    m = _m()
    g = torch.Generator().manual_seed(M + E)
    logits = (torch.randn(M, E, generator=g) * 2).to(dtype)  # (bf16: many equal logits)
    check(m, logits, k, renorm=renorm, scale=1.0 if renorm else 2.5)


@pytest.mark.parametrize("M,E,k", SIZES)
@pytest.mark.parametrize("with_bias", [True, False])
def test_sigmoid(M, E, k, with_bias):
    """Scores on a grid of their own (a permutation of E spread logits, biases
    that are multiples of a larger step), so that rounding cannot reorder
    them."""
    m = _m()
    g = torch.Generator().manual_seed(M + E + k)
    grid = torch.logit((torch.arange(E, dtype=torch.float64) + 1) / (E + 1)).float()
    logits = torch.stack([grid[torch.randperm(E, generator=g)] for _ in range(M)])
    bias = torch.randint(0, 3, (E,), generator=g).float() * 2 if with_bias else None
    check(m, logits, k, sigmoid=True, bias=bias)
    check(m, logits, k, sigmoid=True, bias=bias, renorm=False, scale=0.5)


@pytest.mark.parametrize("E", [9, 40, 300, 1500])
def test_masked_rows(E):
    """-inf and NaN are never chosen; rows run out, and one is empty."""
    m = _m()
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(6, E, generator=g)
    logits[0, ::2] = float("-inf")
    logits[1, 3:] = float("-inf")     # three experts left
    logits[2] = float("-inf")         # none
    logits[3, 1] = float("nan")
    logits[4] = -3e38                 # all equal, the type's lowest values
    logits[5] = float("nan")
    ids, w = check(m, logits, 8)
    assert sorted(ids[1, :3].tolist()) == [0, 1, 2] and (ids[1, 3:] == -1).all() and not w[1, 3:].any()
    assert (ids[2] == -1).all() and not w[2].any() and (ids[5] == -1).all()
    assert ids[4].tolist() == list(range(8))
    ids, w = check(m, logits, 8, renorm=False)
    logits[4] = torch.randn(E, generator=g)
    ids, w = m.route_topk(logits.cuda(), 8, score=m.SCORE_SIGMOID)
    assert (ids[2] == -1).all() and not w[2].any() and (ids[1, 3:] == -1).all()


def test_ties_and_signed_zeros():
    m = _m()
    logits = torch.zeros(3, 70)
    logits[0, ::2] = -0.0
    logits[1, 40:] = 1.0
    ids, w = check(m, logits, 16)
    assert ids[0].tolist() == list(range(16)) and ids[1].tolist() == list(range(40, 56))
    assert torch.allclose(w, torch.full_like(w, 1 / 16))


@pytest.mark.parametrize("E", [100, 600, 1200])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_more_equals_than_the_list_holds(E, sigmoid):
    """Forty equal scores at the edge of the choice, beside clear ones."""
    m = _m()
    g = torch.Generator().manual_seed(E)
    logits = -1.0 - torch.rand(5, E, generator=g).double().mul(64).round().div(16).float()
    at = torch.stack([torch.randperm(E, generator=g)[:44] for _ in range(5)])
    logits.scatter_(1, at[:, :40], torch.full((5, 40), 2.0))
    logits.scatter_(1, at[:, 40:], torch.tensor([3.0, 4.0, 5.0, 6.0]).repeat(5, 1))
    check(m, logits, 16, sigmoid=sigmoid)


@pytest.mark.parametrize("E", [70, 1100])
def test_sigmoid_extremes(E):
    """Scores down to subnormals and zero (logits to -200) order
    as they are, infinite logits score 1."""
    m = _m()
    logits = torch.full((3, E), -200.0)  # 1 / inf: a score of 0, all equal
    logits[0, 5:10] = torch.tensor([-100.0, -95.0, -90.0, -88.0, -86.0])
    logits[1, 7] = float("inf")
    logits[1, 3] = 0.0
    logits[2, 11] = -80.0
    ids, w = m.route_topk(logits.cuda(), 8, score=m.SCORE_SIGMOID, renormalize=False)
    # exp(90) and above overflow FP32: their score is 0, ties to the lowest index
    assert ids[0].tolist() == [9, 8, 0, 1, 2, 3, 4, 5]
    assert ids[1].tolist() == [7, 3, 0, 1, 2, 4, 5, 6]
    assert ids[2].tolist() == [11, 0, 1, 2, 3, 4, 5, 6]
    assert w[1, :2].tolist() == [1.0, 0.5] and not w[1, 2:].any()


def test_strided_logits_and_the_layer():
    """Rows with a stride; the ids and weights go into the layer as they are."""
    m = _m()
    from workload import gen
    wl = gen.make_workload("tiny_decode", device="cuda", M=4)
    big = torch.randn(4, wl.E + 5, device="cuda")
    logits = big[:, 2:2 + wl.E]
    ids, w = m.route_topk(logits, wl.top_k)
    want_ids, _ = want(logits.cpu(), wl.top_k, False, None, True, 1.0)
    assert torch.equal(ids.cpu(), want_ids)
    pw = m.prepare_weights(wl.weights, wl.E, wl.H, wl.I, wl.fmt)
    ws = m.alloc_workspace(4, wl.E, wl.H, wl.I, wl.top_k, wl.fmt)
    assert torch.isfinite(m.forward(wl.x, pw, ids, w, workspace=ws)).all()
    assert m.route_topk(logits[:0], 2)[0].shape == (0, 2)


def test_refusals():
    m = _m()
    l = torch.zeros(3, 20, device="cuda")
    with pytest.raises(TypeError):
        m.route_topk(l.half(), 2)
    with pytest.raises(ValueError):
        m.route_topk(l.cpu(), 2)
    with pytest.raises(ValueError):
        m.route_topk(l.t(), 2)
    with pytest.raises(ValueError):
        m.route_topk(l, 0)
    with pytest.raises(ValueError):
        m.route_topk(l, 2, score=m.SCORE_SIGMOID, bias=torch.zeros(19, device="cuda"))
    for bad in (lambda: m.route_topk(l, 17), lambda: m.route_topk(l[:, :4], 5), lambda: m.route_topk(l, 2, score=7),
                lambda: m.route_topk(l, 2, bias=torch.zeros(20, device="cuda")),
                lambda: m.route_topk(l, 2, scale=float("nan"))):
        with pytest.raises(m.MoeFp4Error):
            bad()
