"""Gated activations in front of the FP8 quantiser: what is not finite stays
visible, and every step is the operation that its definition names.

Finite values: half an E4M3 step of the value (1/16 of it, or 2^-10 scales
below the normals) and 2^-12 of the block's largest for the FP32 activation
and scale."""
import pytest
import torch

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
ALPHA, BETA, LIMIT = 1.702, 1.0, 3.0


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def quantise(m, x, kind):
    if kind == "oai":
        return m.fp8_quantize(x, act=m.ACT_SWIGLUOAI, alpha=ALPHA, beta=BETA, limit=LIMIT)
    return m.fp8_quantize(x, act=m.ACT_SILU if kind == "silu" else m.ACT_GELU_TANH)


def activation_64(gate, up, kind):
    if kind == "silu":
        return gate * torch.sigmoid(gate) * up
    if kind == "gelu":
        return 0.5 * gate * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (gate + 0.044715 * gate ** 3))) * up
    g, u = gate.clamp(max=LIMIT), up.clamp(-LIMIT, LIMIT)  # (clamp hands NaN on)
    return (u + BETA) * g * torch.sigmoid(ALPHA * g)


@pytest.mark.parametrize("rows", [9, 3000])  # (the two forms of the kernel)
@pytest.mark.parametrize("kind", ["silu", "gelu", "oai"])
def test_what_is_not_finite_stays_visible(rows, kind):
    """One special gate or up a row: NaN wherever the activation is NaN, an
    infinite scale with NaN and zeros where it is infinite, and no effect on
    other elements, blocks and rows."""
    m = _m()
    K = 272
    special = [("gate", NAN), ("up", NAN), ("gate", INF), ("gate", -INF), ("up", INF), ("up", -INF)]
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, 2 * K, generator=g) * 2).to(torch.bfloat16)
    for i, (where, value) in enumerate(special):
        x[i, 130 + i + (K if where == "up" else 0)] = value
    q, s = quantise(m, x.cuda(), kind)
    v = activation_64(x[:, :K].double(), x[:, K:].double(), kind)
    s64 = s.cpu().double().repeat_interleave(128, 1)[:, :K]
    got = q.cpu().double()
    want_nan = torch.isnan(v) | torch.isinf(v)  # (an infinity over an infinite scale)
    assert torch.equal(torch.isnan(got), want_nan)
    assert torch.equal(torch.isinf(s.cpu()), torch.nn.functional.pad(torch.isinf(v), (0, 112)).view(rows, 3, 128).any(2))
    beside = torch.isinf(s64) & ~want_nan
    assert not got[beside].any()
    fine = ~want_nan & ~beside
    err, bound = (got * s64 - v).abs(), v.abs() / 16 + s64 * 2.0 ** -10 + 448 * s64 * 2.0 ** -12
    assert (err <= bound)[fine].all()


@pytest.mark.parametrize("rows", [1024, 65536])
@pytest.mark.parametrize("alpha,limit", [(1.702, 7.0), (0.25, 256.0)])
def test_swiglu_oai_precision(rows, alpha, limit):
    """The clamped SwiGLU of every BF16 gate, alone in its row, through its
    scale. With x = alpha g: the product is off by 2^-24 of itself, which the
    exponential turns into |x| 2^-24, and the hardware's exponential is
    documented to be off by at most 2 + 1.173 |x| units of 2^-23; the sum, the
    product, the quotient and the scale add less than 2^-21. Where e^-x leaves
    FP32 (|x| > 85) or the value does, there is nothing to compare."""
    m = _m()
    g = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    x = torch.zeros(65536, 32, dtype=torch.bfloat16, device="cuda")
    x[:, 5], x[:, 21] = g, 0.75
    got = torch.cat([m.fp8_quantize(c, act=m.ACT_SWIGLUOAI, alpha=alpha, beta=BETA, limit=limit)[1]
                     for c in x.split(rows)])[:, 0].double()
    f = g.double().clamp(max=limit)
    alpha = torch.tensor(alpha, dtype=torch.float32).double().item()
    e = alpha * f
    want = (1.75 * f * torch.sigmoid(e)).abs() / 448
    fine = (e.abs() <= 85) & (want > 2.0 ** -125)
    assert fine.sum() > 30000
    bound = ((2 + 1.173 * e.abs()) * 2.0 ** -23 + e.abs() * 2.0 ** -24 + 2.0 ** -21) * want
    assert ((got - want).abs() <= bound)[fine].all()
