"""Host-side checks of the operators around the layer (no GPU needed): the
entry points reject bad arguments with the documented status codes before
they touch the GPU, take empty batches, and size their workspace."""
import ctypes

import pytest

from fp4_weight_moe_gb300 import _capi
from fp4_weight_moe_gb300 import build as build_mod

OK, EINVAL, EUNSUPPORTED, EWORKSPACE = (_capi.MOE_FP4_OK, _capi.MOE_FP4_EINVAL, _capi.MOE_FP4_EUNSUPPORTED,
                                        _capi.MOE_FP4_EWORKSPACE)
P = 0x10000  # never dereferenced: every call here is refused, or empty


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return _capi.lib()


def quantize(x=P, x_row=None, act=None, q=P, q_row=None, s=P, s_row=1, s_block=4, M=4, K=256):
    a = None if act is None else ctypes.byref(act)
    wide = 1 if act is None else 2
    return _capi.lib().moe_fp4_fp8_quantize(x, wide * K if x_row is None else x_row, a, q, K if q_row is None else q_row,
                                            s, s_row, s_block, M, K, None)


def test_quantize_arguments():
    silu = _capi.MoeFp4Activation(_capi.MOE_FP4_ACT_SILU, 0.0, 0.0, 0.0)
    assert quantize(M=0) == OK and quantize(M=0, act=silu) == OK
    assert quantize(K=24) == EUNSUPPORTED
    for bad in (dict(M=-1), dict(K=0), dict(x=0), dict(q=0), dict(s=0), dict(x=P + 8), dict(q=P + 8), dict(s=P + 2),
                dict(x_row=128), dict(x_row=260), dict(q_row=128), dict(q_row=264), dict(s_row=-1), dict(s_block=-4),
                dict(act=silu, x_row=256), dict(act=_capi.MoeFp4Activation(_capi.MOE_FP4_ACT_RELU2, 0.0, 0.0, 0.0)),
                dict(act=_capi.MoeFp4Activation(9, 0.0, 0.0, 0.0)),
                dict(act=_capi.MoeFp4Activation(_capi.MOE_FP4_ACT_SWIGLUOAI, 1.7, 1.0, 0.0)),
                dict(act=_capi.MoeFp4Activation(_capi.MOE_FP4_ACT_SWIGLUOAI, float("nan"), 1.0, 7.0))):
        assert quantize(**bad) == EINVAL, bad


def matmul(x=P, x_row=None, xs=P, xs_row=1, xs_block=4, w=P, w_row=None, ws=P, ws_row=2, add=0, add_row=0, out=P,
           out_row=None, f32=0, M=4, N=96, K=256):
    return _capi.lib().moe_fp4_fp8_matmul(x, K if x_row is None else x_row, xs, xs_row, xs_block, w,
                                          K if w_row is None else w_row, ws, ws_row, add, add_row, out,
                                          N if out_row is None else out_row, f32, M, N, K, None)


def linear(x=P, x_row=None, w=P, ws=P, ws_row=2, add=0, add_row=0, out=P, M=64, N=96, K=256, wsp=P, wsb=1 << 20):
    return _capi.lib().moe_fp4_fp8_linear(x, K if x_row is None else x_row, w, K, ws, ws_row, add, add_row, out, N, 0,
                                          M, N, K, wsp, wsb, None)


def test_product_arguments():
    assert matmul(M=0) == OK and linear(M=0) == OK
    assert matmul(K=264) == EUNSUPPORTED and linear(K=264) == EUNSUPPORTED
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(x=0), dict(xs=0), dict(w=0), dict(ws=0), dict(out=0),
                dict(x=P + 8), dict(w=P + 8), dict(out=P + 1), dict(out=P + 2, f32=1), dict(f32=2), dict(x_row=128),
                dict(x_row=264), dict(w_row=128), dict(w_row=264), dict(ws_row=1, N=200), dict(out_row=95),
                dict(add=P, add_row=95), dict(add=P + 1, add_row=96), dict(xs_row=-1), dict(xs_block=-1)):
        assert matmul(**bad) == EINVAL, bad
    assert matmul(M=1 << 30, N=1 << 30) == EUNSUPPORTED  # tile numbers past 32 bits
    for bad in (dict(x=0), dict(x=P + 8), dict(x_row=260), dict(x_row=128), dict(add=P, add_row=5)):
        assert linear(**bad) == EINVAL, bad


def test_linear_workspace():
    size = _capi.moe_fp4_fp8_linear_workspace_bytes
    assert size(64, 256) == 64 * 256 + 64 * 2 * 4
    assert size(3, 272) == 1024 + 256 and size(-1, 256) == 0 and size(4, 24) == 0 and size(4, 0) == 0
    assert linear(wsp=0) == EWORKSPACE and linear(wsp=P + 16) == EWORKSPACE and linear(wsb=100) == EWORKSPACE
    # a workspace that is given must be large enough even where it is not needed
    assert linear(M=4, wsb=16) == EWORKSPACE


def norm(**kw):
    a = _capi.MoeFp4BlockNormArgs()
    args = dict(residual=P, residual_row=64, w_pre=P, normed=P, normed_row=64, scale=1.0, eps=1e-6, M=4, H=64)
    args.update(kw)
    for k, v in args.items():
        setattr(a, k, v)
    return _capi.lib().moe_fp4_block_norm(bytes(a), None)


def test_block_norm_arguments():
    assert norm(M=0) == OK and _capi.lib().moe_fp4_block_norm(None, None) == EINVAL
    assert norm(H=32769) == EUNSUPPORTED
    q = dict(q=P, q_row=64, s=P, s_row=1, s_block=4)
    assert norm(**q, H=72, residual_row=72, normed_row=72) == EUNSUPPORTED  # H % 16
    b = dict(block_out=P, block_row=64)
    for bad in (dict(M=-1), dict(H=0), dict(residual=0), dict(residual=P + 1), dict(residual=P + 2, residual_f32=1),
                dict(w_pre=0), dict(normed=0), dict(normed_row=32), dict(scale=float("inf")), dict(eps=-1e-6),
                dict(eps=float("nan")), dict(offset=float("inf")), dict(residual_row=-64),
                dict(residual_out=P, residual_out_row=63), dict(w_pre=0, normed=0),
                dict(w_pre=P + 2, weights_f32=1), dict(**q | dict(s=0)), dict(**q | dict(q_row=32)),
                dict(**q | dict(q=P + 8)), dict(**q, residual=P + 2), dict(**b | dict(block_row=-1)),
                dict(**b, gate=P, gate_col=2), dict(**b, gate=P, gate_row=-1, gate_col=1),
                dict(**b, gate=P + 2, gate_f32=1, gate_col=1)):
        assert norm(**bad) == EINVAL, bad


def test_block_norm_pack_matches_the_struct():
    """The packed bytes are those of a filled structure, field by field."""
    values = [i + 1 for i in range(18)] + [0.5, 0.25, 2.0] + [1, 0, 1, 7, 9]
    assert _capi.MoeFp4BlockNormArgs.PACK.pack(*values) == bytes(_capi.MoeFp4BlockNormArgs(*values))


def topk(l=P, row=64, f32=1, bias=0, score=0, renorm=1, scale=1.0, ids=P, w=P, M=4, E=64, k=4):
    return _capi.lib().moe_fp4_route_topk(l, row, f32, bias, score, renorm, scale, ids, w, M, E, k, None)


def test_route_topk_arguments():
    assert topk(M=0) == OK
    for bad in (dict(k=17), dict(k=65, E=64), dict(E=3), dict(E=65537, row=65537)):
        assert topk(**bad) == EUNSUPPORTED, bad
    for bad in (dict(M=-1), dict(E=0), dict(k=0), dict(score=2), dict(score=-1), dict(bias=P), dict(scale=float("nan")),
                dict(l=0), dict(ids=0), dict(w=0), dict(row=-1), dict(l=P + 2), dict(l=P + 1, f32=0),
                dict(bias=P + 2, score=1), dict(ids=P + 2), dict(w=P + 2)):
        assert topk(**bad) == EINVAL, bad


def test_status_arguments():
    assert _capi.lib().moe_fp4_fp8_status(None, 0, None) == EINVAL
