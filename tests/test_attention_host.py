"""Host-side checks of the operators on a paged cache (no GPU needed): the
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


def call(fn, struct, defaults, changes):
    a = struct()
    for k, v in (defaults | changes).items():
        setattr(a, k, v)
    return getattr(_capi.lib(), fn)(bytes(a), None)


STEP = dict(lengths=P, new_tokens=P, tables=P, table_row=8, free_pages=P, free_count=P, offsets=P, positions=P, slots=P,
            lengths_out=P, free_count_out=P, accepted=P, table_width=8, free_capacity=100, page_size=16, R=4, tokens=4)


def step(**kw):
    return call("moe_fp4_cache_step", _capi.MoeFp4CacheStepArgs, STEP, kw)


def test_step_arguments():
    for bad in (dict(R=-1), dict(tokens=-1), dict(table_width=-1), dict(free_capacity=-1), dict(lengths=0),
                dict(new_tokens=0), dict(tables=0), dict(table_row=7), dict(free_pages=0), dict(free_count=0),
                dict(offsets=0), dict(positions=0), dict(slots=0), dict(lengths_out=0), dict(free_count_out=0),
                dict(accepted=0), dict(lengths=P + 2), dict(slots=P + 4), dict(tables=P + 1), dict(accepted=P + 2)):
        assert step(**bad) == EINVAL, bad
    for bad in (dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(page_size=0), dict(R=65537)):
        assert step(**bad) == EUNSUPPORTED, bad
    assert _capi.lib().moe_fp4_cache_step(None, None) == EINVAL


ROPE = dict(q_in=P, k_in=P, v_in=P, q_row=1024, q_head=128, k_row=256, k_head=128, v_row=256, v_head=128, w_q=P, w_k=P,
            rotary=P, positions=P, q_out=P, k_out=P, q_out_row=1024, q_out_head=128, k_out_row=256, k_out_head=128,
            cache=P, slots=P, eps=1e-6, offset=0.0, k_scale=1.0, v_scale=1.0, weights_f32=0, interleaved=0,
            positions_i64=0, positions_max=100, T=4, Hq=8, Hkv=2, D=128, rot=128, pages=10, page_size=16)


def rope(**kw):
    return call("moe_fp4_qk_norm_rope", _capi.MoeFp4QkNormRopeArgs, ROPE, kw)


def test_rope_arguments():
    assert rope(T=0) == OK and rope(T=0, q_in=0, slots=0) == OK and rope(T=0, cache=0) == OK
    for bad in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(rot=-16), dict(q_in=0), dict(k_in=0), dict(v_in=0),
                dict(q_out=0), dict(slots=0), dict(q_in=P + 8), dict(k_in=P + 2), dict(v_in=P + 8), dict(q_out=P + 8),
                dict(q_row=1020), dict(q_head=4), dict(k_row=-256), dict(v_head=-8), dict(q_out_row=1016),
                dict(q_out_head=120), dict(cache=P + 8), dict(slots=P + 4), dict(positions=0),
                dict(positions=P + 2), dict(positions=P + 4, positions_i64=1), dict(positions_max=0),
                dict(rotary=P + 8), dict(rot=0), dict(w_q=P + 2), dict(w_k=P + 8), dict(eps=-1.0),
                dict(eps=float("nan")), dict(offset=float("inf")), dict(k_scale=0.0), dict(v_scale=-1.0),
                dict(k_scale=float("inf")), dict(v_scale=float("nan")), dict(pages=0), dict(cache=0, k_out=0),
                dict(cache=0, k_out_row=248)):
        assert rope(**bad) == EINVAL, bad
    for bad in (dict(D=96), dict(D=512), dict(rot=24), dict(rot=144), dict(page_size=8), dict(Hq=65536)):
        assert rope(**bad) == EUNSUPPORTED, bad


def read(cache=P, pages=10, page_size=16, Hkv=2, D=128, slots=P, ks=1.0, vs=1.0, k=P, v=P, T=4):
    return _capi.lib().moe_fp4_cache_read(cache, pages, page_size, Hkv, D, slots, ks, vs, k, v, T, None)


def test_read_arguments():
    assert read(T=0) == OK
    for bad in (dict(T=-1), dict(Hkv=0), dict(pages=0), dict(cache=0), dict(slots=0), dict(k=0), dict(v=0),
                dict(cache=P + 8), dict(slots=P + 4), dict(k=P + 8), dict(v=P + 2), dict(ks=0.0), dict(vs=float("inf"))):
        assert read(**bad) == EINVAL, bad
    for bad in (dict(D=32), dict(D=192), dict(page_size=24)):
        assert read(**bad) == EUNSUPPORTED, bad


ATTN = dict(q=P, q_row=1024, q_head=128, cache=P, tables=P, table_row=8, lengths=P, offsets=P, sinks=0, out=P,
            out_row=1024, out_head=128, lse=0, workspace=P, workspace_bytes=1 << 40, scale=0.1, k_scale=1.0, v_scale=1.0,
            window=0, T=4, R=2, Hq=8, Hkv=2, D=128, pages=10, page_size=16, table_width=8)


def attention(**kw):
    return call("moe_fp4_attention", _capi.MoeFp4AttentionArgs, ATTN, kw)


def test_attention_arguments():
    assert attention(T=0) == OK and attention(T=0, workspace=0) == OK
    for bad in (dict(T=-1), dict(R=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(q=0), dict(out=0), dict(cache=0),
                dict(tables=0), dict(lengths=0), dict(offsets=0), dict(q=P + 8), dict(out=P + 8), dict(cache=P + 8),
                dict(q_row=1020), dict(q_head=12), dict(q_row=-1024), dict(out_row=1016), dict(out_head=64),
                dict(table_row=7), dict(table_width=-1), dict(window=-1), dict(scale=float("nan")),
                dict(k_scale=0.0), dict(v_scale=float("inf")), dict(pages=0), dict(lse=P + 2), dict(sinks=P + 2),
                dict(lengths=P + 2), dict(offsets=P + 1), dict(tables=P + 2)):
        assert attention(**bad) == EINVAL, bad
    for bad in (dict(D=96), dict(Hq=9), dict(Hq=130, q_row=16640, out_row=16640), dict(R=65537), dict(page_size=20),
                dict(table_width=1 << 27, table_row=1 << 27)):
        assert attention(**bad) == EUNSUPPORTED, bad
    # a table whose last step of tokens would pass 32 bits, and the widest that does not
    for width, page in (((1 << 27) - 1, 16), ((1 << 24) - 1, 128)):
        assert attention(table_width=width, table_row=width, page_size=page) == EUNSUPPORTED
    assert attention(table_width=(1 << 27) - 64, table_row=1 << 27, T=0) == OK
    # heads within rows, or rows within heads
    assert attention(out_row=128, out_head=504) == EINVAL
    for bad in (dict(workspace=0), dict(workspace=P + 16), dict(workspace_bytes=64)):
        assert attention(**bad) == EWORKSPACE, bad


def test_attention_workspace():
    size = _capi.moe_fp4_attention_workspace_bytes
    assert size(1, 8, 2, 128) > 0 and size(100000, 8, 2, 128) == 0 and size(-1, 8, 2, 128) == 0
    assert size(4, 9, 2, 128) == 0 and size(4, 8, 2, 96) == 0
    assert size(512, 8, 2, 128) >= size(1, 8, 2, 128)


def test_status_arguments():
    assert _capi.lib().moe_fp4_attention_status(None, 0, None) == EINVAL


@pytest.mark.parametrize("struct", [_capi.MoeFp4CacheStepArgs, _capi.MoeFp4QkNormRopeArgs, _capi.MoeFp4AttentionArgs])
def test_packs_match_the_structs(struct):
    """The packed bytes are those of a filled structure, field by field."""
    values = [i + 1 for i in range(len(struct._fields_))]
    assert struct.PACK.pack(*values) == bytes(struct(*values))
    assert ctypes.sizeof(struct) == struct.PACK.size
