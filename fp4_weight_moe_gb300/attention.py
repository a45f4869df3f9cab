"""The attention's side of a served block, over a paged cache in 4 bits:

* ``cache_step``      pages for a step's new tokens and where each of them goes
                      (block tables, slots, positions), from the lengths of the
                      requests;
* ``qk_norm_rope``    norms of queries and keys for each head and the rotation
                      by their positions, the keys and values stored in the
                      cache or the keys handed on;
* ``fp4_attention``   attention of new tokens over the cache;
* ``fp4_cache_read``  what the cache holds, as BF16.

Thin wrappers of the C entry points of include/moe_fp4.h, as those of ``ops``:
they check types and shapes, allocate outputs, and launch on the current
stream (or ``stream``).
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from . import _capi
from .ops import _BF16, _F32, _INT_MAX, _current_device, _device, _empty, _fail, _float_type, _on, _raw_stream, _vector

_I32, _I64, _U8, _BOOL = torch.int32, torch.int64, torch.uint8, torch.bool
_PACK_STEP = _capi.MoeFp4CacheStepArgs.PACK.pack
_PACK_ROPE = _capi.MoeFp4QkNormRopeArgs.PACK.pack
_PACK_ATTENTION = _capi.MoeFp4AttentionArgs.PACK.pack
CACHE_BLOCK = 16  # tokens of a page whose keys and values lie together


class CacheStep(NamedTuple):
    """What ``cache_step`` gives."""
    offsets: torch.Tensor     # int32 [R + 1]: new tokens before each request
    positions: torch.Tensor   # int32 [tokens]
    slots: torch.Tensor       # int64 [tokens], -1: not in the cache
    lengths: torch.Tensor     # int32 [R], with the accepted tokens
    free_count: torch.Tensor  # int32 [1]
    accepted: torch.Tensor    # int32 [R]: new tokens, or 0 where the request was refused


# Each call costs the host more than a small kernel costs the GPU: the
# functions below look at the usual arguments in one test, and leave all others
# to these, which find and name what is wrong.
def _heads(t: torch.Tensor, name: str, dev: int, rows=None, heads=None, dim=None):
    """Check a bfloat16 [tokens, heads, D] tensor with contiguous columns;
    returns its strides per token and per head."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be {_BF16}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not cuda:{dev}")
    shape = t.shape
    if len(shape) != 3 or (rows is not None and shape != (rows, heads, dim)):
        raise ValueError(f"{name} must be [{'tokens' if rows is None else rows}, {heads or 'heads'}, {dim or 'D'}], "
                         f"not {list(shape)}")
    row, head, col = t.stride()
    if col != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have contiguous columns")
    # (one token or head has no stride of its own)
    return (row if shape[0] != 1 else shape[1] * shape[2]), (head if shape[1] != 1 else shape[2])


def _cache_sizes(cache: torch.Tensor, dev: int):
    """(pages, heads, page size, D) of a cache."""
    if cache.dtype is not _U8:
        raise TypeError(f"cache must be {_U8}, not {cache.dtype}")
    if cache.get_device() != dev:
        raise ValueError(f"cache is on {cache.device}, not cuda:{dev}")
    if cache.dim() != 5 or cache.shape[3] != 2 or cache.shape[4] % 9 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous [pages, kv_heads, page_size / 16, 2, 9 * D], "
                         f"not {list(cache.shape)}")
    pages, heads, blocks, _, width = cache.shape
    if pages > _INT_MAX:
        raise ValueError(f"cache must have fewer than 2^31 pages, not {pages}")
    return pages, heads, blocks * CACHE_BLOCK, width // 9


def _int_vector(t: torch.Tensor, name: str, dtype, dev: int, n: int) -> int:
    _vector(t, name, dtype, dev, n)
    return t.data_ptr()


def _tables(t: torch.Tensor, dev: int, R: int):
    """(pointer, row stride, width) of block tables."""
    if t.dtype is not _I32:
        raise TypeError(f"tables must be {_I32}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"tables is on {t.device}, not cuda:{dev}")
    if t.dim() != 2 or t.shape[0] != R or t.shape[1] > _INT_MAX:
        raise ValueError(f"tables must be [{R}, pages of a request], not {list(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError("tables must have contiguous columns")
    return t.data_ptr(), (t.stride(0) if R != 1 else t.shape[1]), t.shape[1]


def _step_arguments(lengths, new_tokens, tables, free_pages, free_count, tokens):
    """(table width, its row stride) of cache_step's arguments, checked one by one."""
    dev = _device(lengths)
    if lengths.dim() != 1 or lengths.shape[0] > _INT_MAX:
        raise ValueError(f"lengths must be a vector, not {list(lengths.shape)}")
    if not 0 <= tokens <= _INT_MAX:
        raise ValueError(f"tokens must be in [0, 2^31), not {tokens}")
    R = lengths.shape[0]
    _vector(lengths, "lengths", _I32, dev, R)
    _vector(new_tokens, "new_tokens", _I32, dev, R)
    _, row, width = _tables(tables, dev, R)
    if free_pages.dim() != 1 or free_pages.shape[0] > _INT_MAX:
        raise ValueError(f"free_pages must be a vector, not {list(free_pages.shape)}")
    _vector(free_pages, "free_pages", _I32, dev, free_pages.shape[0])
    _vector(free_count, "free_count", _I32, dev, 1)
    return width, row


def alloc_fp4_cache(pages: int, page_size: int, kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A zeroed cache: uint8 ``[pages, kv_heads, page_size // 16, 2, 9 *
    head_dim]``.  Of each 16 tokens of a head first the keys, then the values,
    each 16 rows of head_dim / 2 bytes (E2M1, the even column in the low
    nibble) and 16 rows of head_dim / 16 scales (E4M3, one per 16 columns).
    page_size 16, 32, 64 or 128; head_dim 64, 128 or 256."""
    if page_size not in (16, 32, 64, 128) or head_dim not in (64, 128, 256):
        raise _capi.MoeFp4Error("alloc_fp4_cache", _capi.MOE_FP4_EUNSUPPORTED)
    return torch.zeros((pages, kv_heads, page_size // CACHE_BLOCK, 2, 9 * head_dim), dtype=_U8,
                       device=device or torch.device("cuda"))


def rotary_table(positions: int, rot_dim: int, theta: float = 10000.0, device=None) -> torch.Tensor:
    """float32 ``[positions, rot_dim]`` for ``qk_norm_rope``: the cosines, then
    the sines, of position * theta^(-2 i / rot_dim), from 64 bits."""
    device = device or torch.device("cuda")
    power = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * theta ** -power
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# ------------------------------------------------------------------------ cache
def cache_step(lengths: torch.Tensor, new_tokens: torch.Tensor, tables: torch.Tensor, free_pages: torch.Tensor,
               free_count: torch.Tensor, page_size: int, tokens: int, finished: Optional[torch.Tensor] = None,
               lengths_out: Optional[torch.Tensor] = None, free_count_out: Optional[torch.Tensor] = None,
               stream=None) -> CacheStep:
    """One step of a batch of requests: pages for ``new_tokens [R]`` more
    tokens behind ``lengths [R]``, and where each goes.

    ``tables [R, pages of a request]`` holds each request's pages,
    ``free_pages`` a stack of free ones, of which the first ``free_count [1]``
    count (all int32); both are updated in place.  The pages of requests with
    ``finished [R]`` (bool or uint8) go back on the stack first, and their
    lengths count as 0.  A request whose pages the stack does not hold, after
    what the requests before it asked for, or whose tokens its table row does
    not hold, is refused: it takes no page, its slots are -1, its length stays.
    ``tokens`` rows of positions and slots are given; those behind the last
    new token are 0 and -1.  ``lengths_out`` and ``free_count_out`` may be
    ``lengths`` and ``free_count``."""
    if stream is not None:
        with _on(stream, lengths):
            return cache_step(lengths, new_tokens, tables, free_pages, free_count, page_size, tokens, finished,
                              lengths_out, free_count_out)
    dev, device = lengths.get_device(), lengths.device
    shape, tab_shape, free_shape = lengths.shape, tables.shape, free_pages.shape
    R = shape[0] if shape else -1
    if (dev >= 0 and dev == _current_device() and len(shape) == 1 and len(tab_shape) == 2 and tab_shape[0] == R
            and len(free_shape) == 1 and lengths.dtype is new_tokens.dtype is tables.dtype is free_pages.dtype
            is free_count.dtype is _I32 and new_tokens.shape == shape and free_count.shape == (1,)
            and new_tokens.get_device() == tables.get_device() == free_pages.get_device() == free_count.get_device() == dev
            and lengths.is_contiguous() and new_tokens.is_contiguous() and tables.is_contiguous()
            and free_pages.is_contiguous() and R <= _INT_MAX and tab_shape[1] <= _INT_MAX and free_shape[0] <= _INT_MAX
            and 0 <= tokens <= _INT_MAX):
        width = tab_row = tab_shape[1]
    else:
        width, tab_row = _step_arguments(lengths, new_tokens, tables, free_pages, free_count, tokens)
    p_fin = 0
    if finished is not None:
        _vector(finished, "finished", _U8 if finished.dtype is _U8 else _BOOL, dev, R)
        p_fin = finished.data_ptr()
    if lengths_out is None:
        lengths_out = _empty(R, dtype=_I32, device=device)
    else:
        _vector(lengths_out, "lengths_out", _I32, dev, R)
    if free_count_out is None:
        free_count_out = _empty(1, dtype=_I32, device=device)
    else:
        _vector(free_count_out, "free_count_out", _I32, dev, 1)
    offsets = _empty(R + 1, dtype=_I32, device=device)
    positions = _empty(tokens, dtype=_I32, device=device)
    slots = _empty(tokens, dtype=_I64, device=device)
    accepted = _empty(R, dtype=_I32, device=device)
    st = _capi.lib().moe_fp4_cache_step(
        _PACK_STEP(lengths.data_ptr(), new_tokens.data_ptr(), p_fin, tables.data_ptr(), tab_row, free_pages.data_ptr(),
                   free_count.data_ptr(), offsets.data_ptr(), positions.data_ptr(), slots.data_ptr(),
                   lengths_out.data_ptr(), free_count_out.data_ptr(), accepted.data_ptr(), width, free_shape[0],
                   page_size, R, tokens), _raw_stream(dev))
    if st:
        _fail("moe_fp4_cache_step", st)
    return CacheStep(offsets, positions, slots, lengths_out, free_count_out, accepted)


def fp4_cache_read(cache: torch.Tensor, slots: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """(``k``, ``v``), bfloat16 ``[T, kv_heads, D]``: what ``cache`` holds at
    ``slots [T]`` (int64); zeros for slots that are negative or past it."""
    if stream is not None:
        with _on(stream, cache):
            return fp4_cache_read(cache, slots, k_scale, v_scale)
    dev = _device(cache)
    pages, heads, page_size, D = _cache_sizes(cache, dev)
    shape = slots.shape
    if len(shape) != 1 or shape[0] > _INT_MAX:
        raise ValueError(f"slots must be a vector, not {list(shape)}")
    T = shape[0]
    p_slots = _int_vector(slots, "slots", _I64, dev, T)
    k = _empty((T, heads, D), dtype=_BF16, device=cache.device)
    v = _empty((T, heads, D), dtype=_BF16, device=cache.device)
    st = _capi.lib().moe_fp4_cache_read(cache.data_ptr(), pages, page_size, heads, D, p_slots, k_scale, v_scale,
                                        k.data_ptr(), v.data_ptr(), T, _raw_stream(dev))
    if st:
        _fail("moe_fp4_cache_read", st)
    return k, v


# ------------------------------------------------------------- norms and rotation
def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor] = None,
                 rotary: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, weight_offset: float = 0.0,
                 interleaved: bool = False, v: Optional[torch.Tensor] = None, cache: Optional[torch.Tensor] = None,
                 slots: Optional[torch.Tensor] = None, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Queries ``q [T, heads, D]`` and keys ``k [T, kv_heads, D]`` (bfloat16,
    any strides per token and head, so slices of one projection's output),
    normed per head and rotated by their ``positions [T]`` (int32 or int64):

        y = x * rsqrt(mean(x^2) + eps) * (weight_offset + weight)     (y = x without a weight)
        (a, b) -> (a c - b s, b c + a s)

    ``rotary`` (``rotary_table``: float32 ``[positions, rot]``) holds c, then s,
    for the first rot columns, paired as i and i + rot / 2, or, ``interleaved``,
    2 i and 2 i + 1; without it nothing is rotated.  Weights ``[D]`` are both
    bfloat16 or both float32.

    Returns ``(q', k')`` in bfloat16.  With a ``cache`` (``alloc_fp4_cache``),
    ``v [T, kv_heads, D]`` and ``slots [T]`` (int64; -1: not stored), k' and v
    go there in 4 bits instead, divided by ``k_scale`` and ``v_scale``, and
    k' is None.  (Keys without a weight are computed twice on their way there:
    8192 tokens of 32 and 8 heads of 128 in 58 us, with one in 46.)"""
    if stream is not None:
        with _on(stream, q):
            return qk_norm_rope(q, k, positions, rotary, q_weight, k_weight, eps, weight_offset, interleaved, v, cache,
                                slots, k_scale, v_scale)
    dev = _device(q)
    shape, k_shape = q.shape, k.shape
    if (len(shape) == 3 and len(k_shape) == 3 and q.dtype is k.dtype is _BF16 and k.get_device() == dev
            and shape[0] == k_shape[0] and shape[2] == k_shape[2] and q.stride(2) == 1 and k.stride(2) == 1
            and shape[0] <= _INT_MAX and shape[1] <= _INT_MAX and k_shape[1] <= _INT_MAX and shape[2] <= _INT_MAX):
        T, Hq, D = shape
        Hkv = k_shape[1]
        q_row, q_head, _ = q.stride()
        k_row, k_head, _ = k.stride()
        if T == 1:  # (has no stride of its own)
            q_row = k_row = 0
        if Hq == 1:
            q_head = 0
        if Hkv == 1:
            k_head = 0
    else:
        q_row, q_head = _heads(q, "q", dev)
        T, Hq, D = shape
        if len(k_shape) != 3:
            raise ValueError(f"k must be [{T}, heads, {D}], not {list(k_shape)}")
        Hkv = k_shape[1]
        k_row, k_head = _heads(k, "k", dev, T, Hkv, D)
        if T > _INT_MAX or Hq > _INT_MAX or Hkv > _INT_MAX or D > _INT_MAX:
            raise ValueError(f"q and k must have fewer than 2^31 tokens, heads and columns, not {list(shape)}")
    p_v = v_row = v_head = p_rot = p_pos = p_cache = p_slots = p_k = w_f32 = 0
    pos64 = places = rot = pages = page_size = 0
    p_wq = p_wk = 0
    if q_weight is not None:
        dtype = _float_type(q_weight, "q_weight")
        _vector(q_weight, "q_weight", dtype, dev, D)
        p_wq, w_f32 = q_weight.data_ptr(), 1 if dtype is _F32 else 0
    if k_weight is not None:
        dtype = _float_type(k_weight, "k_weight")
        if q_weight is not None and dtype is not q_weight.dtype:
            raise TypeError(f"k_weight must be {q_weight.dtype}, as q_weight, not {dtype}")
        _vector(k_weight, "k_weight", dtype, dev, D)
        p_wk, w_f32 = k_weight.data_ptr(), 1 if dtype is _F32 else 0
    if rotary is not None:
        if positions is None:
            raise ValueError("rotary needs positions")
        if rotary.dtype is not _F32:
            raise TypeError(f"rotary must be {_F32}, not {rotary.dtype}")
        if rotary.get_device() != dev or rotary.dim() != 2 or not rotary.is_contiguous() or rotary.shape[0] > _INT_MAX:
            raise ValueError(f"rotary must be a contiguous [positions, rot] on cuda:{dev}, not {list(rotary.shape)} on "
                             f"{rotary.device}")
        places, rot = rotary.shape
        if rot % 16 or rot > D or rot == 0:
            _fail("moe_fp4_qk_norm_rope", _capi.MOE_FP4_EUNSUPPORTED)
        pos64 = 1 if positions.dtype is _I64 else 0
        p_pos = _int_vector(positions, "positions", _I64 if pos64 else _I32, dev, T)
        p_rot = rotary.data_ptr()
    elif positions is not None:
        raise ValueError("positions need rotary")
    k_out = None
    if cache is not None:
        if v is None or slots is None:
            raise ValueError("a cache needs v and slots")
        v_row, v_head = _heads(v, "v", dev, T, Hkv, D)
        pages, heads, page_size, width = _cache_sizes(cache, dev)
        if (heads, width) != (Hkv, D):
            raise ValueError(f"the cache has {heads} heads of {width} columns, k {Hkv} of {D}")
        p_slots = _int_vector(slots, "slots", _I64, dev, T)
        p_v, p_cache = v.data_ptr(), cache.data_ptr()
    elif v is not None or slots is not None:
        raise ValueError("v and slots need a cache")
    else:
        k_out = _empty((T, Hkv, D), dtype=_BF16, device=q.device)
        p_k = k_out.data_ptr()
    q_out = _empty((T, Hq, D), dtype=_BF16, device=q.device)
    st = _capi.lib().moe_fp4_qk_norm_rope(
        _PACK_ROPE(q.data_ptr(), k.data_ptr(), p_v, q_row, q_head, k_row, k_head, v_row, v_head, p_wq, p_wk, p_rot,
                   p_pos, q_out.data_ptr(), p_k, Hq * D, D, Hkv * D, D, p_cache, p_slots, eps, weight_offset, k_scale,
                   v_scale, w_f32, 1 if interleaved else 0, pos64, places, T, Hq, Hkv, D, rot, pages, page_size),
        _raw_stream(dev))
    if st:
        _fail("moe_fp4_qk_norm_rope", st)
    return q_out, k_out


# -------------------------------------------------------------------- attention
def alloc_fp4_attention_workspace(R_max: int, heads: int, kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A workspace for ``fp4_attention(..., workspace=...)`` of up to R_max
    requests: 20 (head_dim 64) to 41 MB, however many they are."""
    n = _capi.moe_fp4_attention_workspace_bytes(R_max, heads, kv_heads, head_dim)
    if n == 0:
        raise _capi.MoeFp4Error("moe_fp4_attention_workspace_bytes", _capi.MOE_FP4_EUNSUPPORTED)
    return torch.empty(n, dtype=_U8, device=device or torch.device("cuda"))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(R: int, heads: int, kv_heads: int, D: int, dev: int) -> int:
    return _capi.moe_fp4_attention_workspace_bytes(R, heads, kv_heads, D)


def _attention_arguments(q, cache, tables, lengths, offsets, window):
    """Sizes and strides of fp4_attention's arguments, checked one by one."""
    dev = _device(q)
    q_row, q_head = _heads(q, "q", dev)
    T, Hq, D = q.shape
    if T > _INT_MAX or Hq > _INT_MAX:
        raise ValueError(f"q must have fewer than 2^31 tokens and heads, not {list(q.shape)}")
    pages, Hkv, page_size, width = _cache_sizes(cache, dev)
    if width != D:
        raise ValueError(f"the cache has heads of {width} columns, q of {D}")
    if lengths.dim() != 1 or lengths.shape[0] >= _INT_MAX:
        raise ValueError(f"lengths must be a vector, not {list(lengths.shape)}")
    R = lengths.shape[0]
    _vector(lengths, "lengths", _I32, dev, R)
    _vector(offsets, "offsets", _I32, dev, R + 1)
    _, tab_row, tab_width = _tables(tables, dev, R)
    if not 0 <= window <= _INT_MAX:
        raise ValueError(f"window must be in [0, 2^31), not {window}")
    return T, Hq, D, q_row, q_head, pages, Hkv, page_size, R, tab_width, tab_row


def fp4_attention(q: torch.Tensor, cache: torch.Tensor, tables: torch.Tensor, lengths: torch.Tensor,
                  offsets: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                  sinks: Optional[torch.Tensor] = None, k_scale: float = 1.0, v_scale: float = 1.0,
                  out: Optional[torch.Tensor] = None, return_lse: bool = False,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Causal attention of new tokens over the cache.

    Request r has ``lengths[r]`` tokens in ``cache`` (its new ones among them)
    on the pages of ``tables[r]``; its queries are the rows ``offsets[r] ..
    offsets[r + 1]`` of ``q [T, heads, D]`` (bfloat16, any strides per token
    and head), for its last tokens.  The query at position p sees the keys j
    with ``p - window < j <= p`` (``window`` 0: all j <= p):

        x_j = scale * k_scale * q . k_j          (scale: 1 / sqrt(D) if None)
        out = v_scale * sum_j e^x_j v_j / (sum_j e^x_j + e^sinks[h])

    ``sinks`` float32 ``[heads]`` or None.  Returns ``out`` bfloat16 ``[T,
    heads, D]``, and with ``return_lse`` ``(out, lse)``, the logarithm of that
    divisor, float32 ``[T, heads]``.  Queries that see no key, and rows of q
    behind the last sequence, get 0 (and sinks[h] or -inf; behind the last
    sequence -inf).  ``workspace`` (alloc_fp4_attention_workspace) is scratch;
    without one the call takes it, 20 to 41 MB, from torch's allocator.

    One kernel serves a call, chosen by its mean number of rows (T * heads /
    kv_heads / R): single tokens beside a prompt's chunk, or padded by many
    rows of q, run up to three times as long as in calls of their own."""
    if stream is not None:
        with _on(stream, q):
            return fp4_attention(q, cache, tables, lengths, offsets, scale, window, sinks, k_scale, v_scale, out,
                                 return_lse, workspace)
    dev, device = q.get_device(), q.device
    shape, c_shape, tab_shape = q.shape, cache.shape, tables.shape
    if (dev >= 0 and dev == _current_device() and len(shape) == 3 and len(c_shape) == 5 and len(tab_shape) == 2
            and q.dtype is _BF16 and cache.dtype is _U8 and tables.dtype is lengths.dtype is offsets.dtype is _I32
            and cache.get_device() == tables.get_device() == lengths.get_device() == offsets.get_device() == dev
            and c_shape[3] == 2 and c_shape[4] == 9 * shape[2] and lengths.shape == (tab_shape[0],)
            and offsets.shape == (tab_shape[0] + 1,) and q.is_contiguous() and cache.is_contiguous()
            and tables.is_contiguous() and lengths.is_contiguous() and offsets.is_contiguous()
            and shape[0] <= _INT_MAX and shape[1] <= _INT_MAX and c_shape[0] <= _INT_MAX and tab_shape[0] < _INT_MAX
            and tab_shape[1] <= _INT_MAX and 0 <= window <= _INT_MAX):
        T, Hq, D = shape
        q_row, q_head = Hq * D, D
        pages, Hkv, page_size = c_shape[0], c_shape[1], c_shape[2] * CACHE_BLOCK
        R, tab_width = tab_shape
        tab_row = tab_width
    else:
        T, Hq, D, q_row, q_head, pages, Hkv, page_size, R, tab_width, tab_row = _attention_arguments(
            q, cache, tables, lengths, offsets, window)
    p_sinks = p_lse = 0
    if sinks is not None:
        _vector(sinks, "sinks", _F32, dev, Hq)
        p_sinks = sinks.data_ptr()
    if out is None:
        out = _empty(shape, dtype=_BF16, device=device)
        out_row, out_head = Hq * D, D
    else:
        out_row, out_head = _heads(out, "out", dev, T, Hq, D)
    lse = None
    if return_lse:
        lse = _empty((T, Hq), dtype=_F32, device=device)
        p_lse = lse.data_ptr()
    if workspace is None:
        workspace = _empty(_workspace_bytes(R, Hq, Hkv, D, dev), dtype=_U8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on q's device")
    st = _capi.lib().moe_fp4_attention(
        _PACK_ATTENTION(q.data_ptr(), q_row, q_head, cache.data_ptr(), tables.data_ptr(), tab_row, lengths.data_ptr(),
                        offsets.data_ptr(), p_sinks, out.data_ptr(), out_row, out_head, p_lse, workspace.data_ptr(),
                        workspace.nbytes, D ** -0.5 if scale is None else scale, k_scale, v_scale, window, T, R, Hq, Hkv, D,
                        pages, page_size, tab_width), _raw_stream(dev))
    if st:
        _fail("moe_fp4_attention", st)
    return (out, lse) if return_lse else out


def fp4_attention_status(clear: bool = False, stream=None) -> int:
    """Status word of the attention kernels on the current device: 0, or bits
    of kernel waits that gave up (the outputs since the last clear are not
    valid).  Synchronises the stream."""
    s = torch.cuda.current_stream().cuda_stream if stream is None else \
        stream if isinstance(stream, int) else stream.cuda_stream
    return _capi.moe_fp4_attention_status(clear, s)
