"""The operators around the layer, as a served model calls them between its
residual stream and ``forward``:

* ``block_norm``    the norms before and after a block, its gate and residual
                    scale, and the normed activations' FP8 form, in one launch;
* ``route_topk``    the router's choice of experts from its logits;
* ``fp8_linear``    products with E4M3 weights that have an FP32 scale per
  ``fp8_matmul``    128 x 128 block (the always-on expert, projections), from
  ``fp8_quantize``  BF16 or already quantised activations.

Those of the attention over a paged cache in 4 bits are in ``attention``.

Thin wrappers of the C entry points of include/moe_fp4.h: they check types and
shapes, allocate outputs, and launch on the current stream (or ``stream``).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _capi

SCORE_SOFTMAX, SCORE_SIGMOID = _capi.MOE_FP4_SCORE_SOFTMAX, _capi.MOE_FP4_SCORE_SIGMOID
FP8 = torch.float8_e4m3fn
_BF16, _F32 = torch.bfloat16, torch.float32
_INT_MAX = 2 ** 31 - 1

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty = torch.empty
_PACK_NORM = _capi.MoeFp4BlockNormArgs.PACK.pack


# Each call costs the host as much as a small kernel costs the GPU, so the
# functions below test what they need in few steps and leave it to _matrix,
# _vector and _device to find and name what is wrong.
def _on(stream, t: torch.Tensor):
    """``stream`` (a torch stream or a raw handle) as the current stream: the
    call's outputs and workspace then come from that stream's own pool, never
    from memory that work on another stream may still be using."""
    _device(t)
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=t.device) if isinstance(stream, int) else stream)


def _device(t: torch.Tensor) -> int:
    """The tensor's device index, which must be the current device's."""
    i = t.get_device()
    if i < 0:
        raise ValueError("libmoe_fp4 takes CUDA tensors only (there is no CPU path)")
    if i != _current_device():
        raise ValueError(f"tensors are on {t.device}, the current device is {_current_device()}")
    return i


def _matrix(t: torch.Tensor, name: str, dtype, dev: int, rows: int, cols: int) -> int:
    """Check a [rows, cols] tensor of one type with contiguous columns;
    returns its row stride."""
    if t.dtype is dtype and t.shape == (rows, cols) and t.get_device() == dev and t.is_contiguous():
        return cols
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not cuda:{dev}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], not {list(t.shape)}")
    if t.stride(1) != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous columns")
    return t.stride(0) if rows != 1 else cols  # (one row has no stride of its own)


def _sizes(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {list(t.shape)}")
    shape = t.shape
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:  # (ctypes would pass the low 32 bits on)
        raise ValueError(f"{name} must have fewer than 2^31 rows and columns, not {list(shape)}")
    return shape


def _float_type(t: torch.Tensor, name: str):
    dtype = t.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"{name} must be {_BF16} or {_F32}, not {dtype}")
    return dtype


def _vector(t: torch.Tensor, name: str, dtype, dev: int, n: int):
    if t.dtype is dtype and t.shape == (n,) and t.get_device() == dev and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not cuda:{dev}")
    raise ValueError(f"{name} must be a contiguous vector of {n} values, not {list(t.shape)}")


def _fail(fn: str, status: int):
    raise _capi.MoeFp4Error(fn, status)


@functools.lru_cache(maxsize=64)
def _activation(kind: int, alpha: float, beta: float, limit: float):
    return ctypes.byref(_capi.MoeFp4Activation(kind, alpha, beta, limit))


def _blocks(n: int) -> int:
    return (n + 127) // 128


# ---------------------------------------------------------------- FP8 products
def fp8_quantize(x: torch.Tensor, act: Optional[int] = None, alpha: float = 0.0, beta: float = 1.0,
                 limit: float = 0.0, stream=None):
    """bf16 ``x [M, K]`` -> (``q`` float8_e4m3fn ``[M, K]``, ``s`` float32
    ``[M, ceil(K / 128)]``): a scale max|x| / 448 per row and 128 columns.
    With ``act`` (ACT_SILU, ACT_GELU_TANH, or ACT_SWIGLUOAI with alpha, beta,
    limit) ``x`` is ``[gate | up] [M, 2K]`` and act(gate) * up is quantised.
    ``s`` is laid out block by block (its strides are (1, M))."""
    if stream is not None:
        with _on(stream, x):
            return fp8_quantize(x, act, alpha, beta, limit)
    dev = _device(x)
    M, K = _sizes(x, "x")
    row = _matrix(x, "x", _BF16, dev, M, K)
    if act is not None:
        if K % 2:
            raise ValueError("a gated x has an even number of columns")
        K //= 2
        act = _activation(act, alpha, beta, limit)
    q = _empty((M, K), dtype=FP8, device=x.device)
    s = torch.empty_strided((M, (K + 127) // 128), (1, M), dtype=_F32, device=x.device)
    st = _capi.lib().moe_fp4_fp8_quantize(x.data_ptr(), row, act, q.data_ptr(), K, s.data_ptr(), 1, M, M, K,
                                          _raw_stream(dev))
    if st:
        _fail("moe_fp4_fp8_quantize", st)
    return q, s


def _product_output(addend, out, out_dtype, dev, device, M, N):
    """(addend pointer, its row stride, out, its row stride, whether float32)."""
    add = add_row = 0
    if addend is not None:
        add_row = _matrix(addend, "addend", _BF16, dev, M, N)
        add = addend.data_ptr()
    if out is None:
        out_dtype = out_dtype or _BF16
        if out_dtype is not _BF16 and out_dtype is not _F32:
            raise TypeError(f"out must be {_BF16} or {_F32}, not {out_dtype}")
        out, out_row = _empty((M, N), dtype=out_dtype, device=device), N
    else:
        out_dtype = out_dtype or _float_type(out, "out")
        out_row = _matrix(out, "out", out_dtype, dev, M, N)
        _float_type(out, "out")
    return add, add_row, out, out_row, 1 if out_dtype is _F32 else 0


def fp8_matmul(x_q: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
               out: Optional[torch.Tensor] = None, addend: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """``out [M, N] = x @ w.T (+ addend)`` for E4M3 ``x_q [M, K]`` with scales
    ``x_scale [M, ceil(K / 128)]`` (any strides) and E4M3 ``w [N, K]`` with
    scales ``w_scale [ceil(N / 128), ceil(K / 128)]``; out bfloat16 (default)
    or float32, rounded once after the bfloat16 ``addend [M, N]``."""
    if stream is not None:
        with _on(stream, x_q):
            return fp8_matmul(x_q, x_scale, w, w_scale, out, addend, out_dtype)
    dev = _device(x_q)
    M, K = _sizes(x_q, "x_q")
    N = _sizes(w, "w")[0]
    row = _matrix(x_q, "x_q", FP8, dev, M, K)
    w_row = _matrix(w, "w", FP8, dev, N, K)
    ws_row = _matrix(w_scale, "w_scale", _F32, dev, (N + 127) // 128, (K + 127) // 128)
    if x_scale.dtype is not _F32:
        raise TypeError(f"x_scale must be float32, not {x_scale.dtype}")
    if x_scale.shape != (M, (K + 127) // 128):
        raise ValueError(f"x_scale must be [{M}, {_blocks(K)}], not {list(x_scale.shape)}")
    if x_scale.get_device() != dev:
        raise ValueError(f"x_scale is on {x_scale.device}, not cuda:{dev}")
    xs_row, xs_block = x_scale.stride()
    add, add_row, out, out_row, f32 = _product_output(addend, out, out_dtype, dev, w.device, M, N)
    st = _capi.lib().moe_fp4_fp8_matmul(x_q.data_ptr(), row, x_scale.data_ptr(), xs_row, xs_block, w.data_ptr(),
                                        w_row, w_scale.data_ptr(), ws_row, add, add_row, out.data_ptr(), out_row, f32,
                                        M, N, K, _raw_stream(dev))
    if st:
        _fail("moe_fp4_fp8_matmul", st)
    return out


def alloc_fp8_workspace(M_max: int, K: int, device=None) -> torch.Tensor:
    """A workspace for ``fp8_linear(..., workspace=...)`` of up to M_max rows."""
    n = _capi.moe_fp4_fp8_linear_workspace_bytes(M_max, K)
    if n == 0:
        raise _capi.MoeFp4Error("moe_fp4_fp8_linear_workspace_bytes", _capi.MOE_FP4_EUNSUPPORTED)
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def fp8_linear(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, out: Optional[torch.Tensor] = None,
               addend: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``fp8_matmul`` of the bfloat16 ``x [M, K]``, quantised as
    ``fp8_quantize`` does.  ``workspace`` (alloc_fp8_workspace) holds the
    quantised rows; without one the call takes it from torch's allocator (up
    to 8 rows of at most 16384 columns need none)."""
    if stream is not None:
        with _on(stream, x):
            return fp8_linear(x, w, w_scale, out, addend, out_dtype, workspace)
    dev = _device(x)
    M, K = _sizes(x, "x")
    N = _sizes(w, "w")[0]
    row = _matrix(x, "x", _BF16, dev, M, K)
    w_row = _matrix(w, "w", FP8, dev, N, K)
    ws_row = _matrix(w_scale, "w_scale", _F32, dev, (N + 127) // 128, (K + 127) // 128)
    add, add_row, out, out_row, f32 = _product_output(addend, out, out_dtype, dev, w.device, M, N)
    ws_ptr = ws_bytes = 0
    if workspace is None:
        if M > _capi.MOE_FP4_DECODE_MAX_M or K > 16384:
            workspace = _empty(_capi.moe_fp4_fp8_linear_workspace_bytes(M, K), dtype=torch.uint8, device=x.device)
    elif workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on x's device")
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    st = _capi.lib().moe_fp4_fp8_linear(x.data_ptr(), row, w.data_ptr(), w_row, w_scale.data_ptr(), ws_row, add,
                                        add_row, out.data_ptr(), out_row, f32, M, N, K, ws_ptr, ws_bytes,
                                        _raw_stream(dev))
    if st:
        _fail("moe_fp4_fp8_linear", st)
    return out


def fp8_status(clear: bool = False, stream=None) -> int:
    """Status word of the FP8 products on the current device: 0, or bits of
    kernel waits that gave up (the outputs since the last clear are not
    valid).  Synchronises the stream."""
    s = torch.cuda.current_stream().cuda_stream if stream is None else \
        stream if isinstance(stream, int) else stream.cuda_stream
    return _capi.moe_fp4_fp8_status(clear, s)


# ------------------------------------------------------------------------ norms
def block_norm(residual: torch.Tensor, pre_weight: Optional[torch.Tensor] = None,
               block_out: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6,
               weight_offset: float = 0.0, residual_out: Optional[torch.Tensor] = None, quantize: bool = False,
               stream=None):
    """One step of the residual stream, RMS norms on both sides of a block:

        z  = rms_norm(block_out) * (weight_offset + post_weight)   (z = block_out without post_weight)
        r' = residual + scale * gate * z                           (r' = residual without block_out)
        n  = rms_norm(r') * (weight_offset + pre_weight)

    ``residual [M, H]`` bfloat16 or float32, ``block_out [M, H]`` bfloat16,
    weights ``[H]`` (both bfloat16 or both float32), ``gate`` bfloat16 or
    float32: ``[H]`` per channel, ``[M, 1]`` per token, or ``[M, H]``.
    Returns ``(r', n)``: r' in residual's type (in ``residual_out`` if given,
    which may be ``residual``; residual itself without block_out), n bfloat16
    (None without pre_weight).  With ``quantize``, ``(r', n, q, s)``: n as
    ``fp8_quantize`` gives it."""
    if stream is not None:
        with _on(stream, residual):
            return block_norm(residual, pre_weight, block_out, post_weight, gate, scale, eps, weight_offset,
                              residual_out, quantize)
    dev = _device(residual)
    M, H = _sizes(residual, "residual")
    dtype, device = _float_type(residual, "residual"), residual.device
    row = _matrix(residual, "residual", dtype, dev, M, H)
    b = b_row = w_post = w_pre = g = g_row = g_col = ro = ro_row = n = q_ptr = s_ptr = s_block = 0
    w_f32 = g_f32 = 0
    if pre_weight is not None:
        w_dtype = _float_type(pre_weight, "pre_weight")
        _vector(pre_weight, "pre_weight", w_dtype, dev, H)
        w_pre, w_f32 = pre_weight.data_ptr(), 1 if w_dtype is _F32 else 0
    elif quantize or block_out is None:
        raise ValueError("without pre_weight there is nothing to " + ("quantize" if quantize else "compute"))
    if block_out is not None:
        b_row = _matrix(block_out, "block_out", _BF16, dev, M, H)
        b = block_out.data_ptr()
        if post_weight is not None:
            if pre_weight is None:
                w_dtype = _float_type(post_weight, "post_weight")
                w_f32 = 1 if w_dtype is _F32 else 0
            _vector(post_weight, "post_weight", w_dtype, dev, H)
            w_post = post_weight.data_ptr()
        if gate is not None:
            g_row, g_col = _gate(gate, dev, M, H)
            g, g_f32 = gate.data_ptr(), 1 if gate.dtype is _F32 else 0
    elif post_weight is not None or gate is not None:
        raise ValueError("post_weight and gate need block_out")
    if residual_out is not None:
        ro_row = _matrix(residual_out, "residual_out", dtype, dev, M, H)
        ro = residual_out.data_ptr()
    elif block_out is not None:
        residual_out = _empty((M, H), dtype=dtype, device=device)
        ro, ro_row = residual_out.data_ptr(), H
    else:
        residual_out = residual
    normed = q = s = None
    if pre_weight is not None:
        normed = _empty((M, H), dtype=_BF16, device=device)
        n = normed.data_ptr()
    if quantize:
        q = _empty((M, H), dtype=FP8, device=device)
        s = torch.empty_strided((M, (H + 127) // 128), (1, M), dtype=_F32, device=device)
        q_ptr, s_ptr, s_block = q.data_ptr(), s.data_ptr(), M
    st = _capi.lib().moe_fp4_block_norm(
        _PACK_NORM(residual.data_ptr(), row, b, b_row, w_post, w_pre, g, g_row, g_col, ro, ro_row, n, H, q_ptr, H,
                   s_ptr, 1, s_block, scale, eps, weight_offset, 1 if dtype is _F32 else 0, w_f32, g_f32, M, H),
        _raw_stream(dev))
    if st:
        _fail("moe_fp4_block_norm", st)
    return (residual_out, normed, q, s) if quantize else (residual_out, normed)


def _gate(gate, dev, M, H):
    """(row, column) strides of a gate."""
    _float_type(gate, "gate")
    if gate.get_device() != dev:
        raise ValueError(f"gate is on {gate.device}, not cuda:{dev}")
    if gate.shape == (H,):
        row, col = 0, gate.stride(0)
    elif gate.shape == (M, H):
        row, col = gate.stride()
    elif gate.shape == (M, 1):
        row, col = gate.stride(0), 0
    else:
        raise ValueError(f"gate must be [{H}], [{M}, 1] or [{M}, {H}], not {list(gate.shape)}")
    if col != 0 and col != 1:
        if H != 1:
            raise ValueError("gate must have contiguous columns")
        col = 1
    return row, col


# ----------------------------------------------------------------------- router
def route_topk(logits: torch.Tensor, top_k: int, score: int = SCORE_SOFTMAX, bias: Optional[torch.Tensor] = None,
               renormalize: bool = True, scale: float = 1.0, stream=None):
    """``logits [M, E]`` (bfloat16 or float32) -> (``topk_ids`` int32
    ``[M, top_k]``, ``topk_weights`` float32 ``[M, top_k]``), as ``forward``
    takes them.  SCORE_SOFTMAX chooses by logit; SCORE_SIGMOID by
    sigmoid(logit) + ``bias`` (float32 ``[E]`` or None) and weighs by
    sigmoid(logit).  Equal scores go to the lowest index; experts with a logit
    of -inf or NaN are never chosen, and a row that runs out of experts ends
    in id -1 with weight 0.  With the softmax a logit of +inf comes first and
    makes its row's weights NaN, as torch.softmax does.  ``renormalize``
    divides by the chosen weights' sum; ``scale`` multiplies the weights."""
    if stream is not None:
        with _on(stream, logits):
            return route_topk(logits, top_k, score, bias, renormalize, scale)
    dev = _device(logits)
    M, E = _sizes(logits, "logits")
    dtype = _float_type(logits, "logits")
    row = _matrix(logits, "logits", dtype, dev, M, E)
    b = 0
    if bias is not None:
        _vector(bias, "bias", _F32, dev, E)
        b = bias.data_ptr()
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    ids = _empty((M, top_k), dtype=torch.int32, device=logits.device)
    weights = _empty((M, top_k), dtype=_F32, device=logits.device)
    st = _capi.lib().moe_fp4_route_topk(logits.data_ptr(), row, 1 if dtype is _F32 else 0, b, score,
                                        1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), M, E,
                                        top_k, _raw_stream(dev))
    if st:
        _fail("moe_fp4_route_topk", st)
    return ids, weights
