"""The operators around the layer, as a served model calls them between its
residual stream and ``forward``:

* ``block_norm``    the norms before and after a block, its gate and residual
                    scale, and the normed activations' FP8 form, in one launch;
* ``route_topk``    the router's choice of experts from its logits;
* ``fp8_linear``    products with E4M3 weights that have an FP32 scale per
  ``fp8_matmul``    128 x 128 block (the always-on expert, projections), from
  ``fp8_quantize``  BF16 or already quantised activations.

Thin wrappers of the C entry points of include/moe_fp4.h: they check types and
shapes, allocate outputs, and launch on the current stream (or ``stream``).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _capi

SCORE_SOFTMAX, SCORE_SIGMOID = _capi.MOE_FP4_SCORE_SOFTMAX, _capi.MOE_FP4_SCORE_SIGMOID
FP8 = torch.float8_e4m3fn
_BF16, _F32 = torch.bfloat16, torch.float32

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Launch:
    """Where a call runs: allocations inside ``with`` come from the launch
    stream's own pool, so that a caller's explicit ``stream`` never receives
    memory that work on the current stream may still be using."""

    def __init__(self, t: torch.Tensor, stream):
        if not t.is_cuda:
            raise ValueError("libmoe_fp4 takes CUDA tensors only (there is no CPU path)")
        self.device = t.device
        self._ctx = None
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"tensors are on {t.device}, the current device is {torch.cuda.current_device()}")
        if stream is None:
            self.stream = _raw_stream(t.device.index) if _raw_stream else torch.cuda.current_stream().cuda_stream
        else:
            self.stream = stream if isinstance(stream, int) else stream.cuda_stream
            self._ctx = torch.cuda.stream(stream if not isinstance(stream, int)
                                          else torch.cuda.ExternalStream(stream, device=t.device))

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False


def _matrix(t: torch.Tensor, name: str, dtypes, dev, rows: Optional[int] = None, cols: Optional[int] = None):
    """Check a [rows, cols] tensor with contiguous columns; returns its row
    stride."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {'columns' if cols is None else cols}], "
                         f"not {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not {dev}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous columns")
    return t.stride(0) if t.shape[0] != 1 else t.shape[1]  # (one row has no stride of its own)


def _vector(t: torch.Tensor, name: str, dtypes, dev, n: int):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} values, not {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, not {dev}")


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
    go = _Launch(x, stream)
    row = _matrix(x, "x", (_BF16,), go.device)
    M, K = x.shape
    if act is not None:
        if K % 2:
            raise ValueError("a gated x has an even number of columns")
        K //= 2
        act = _capi.MoeFp4Activation(act, alpha, beta, limit)
    with go:
        q = torch.empty((M, K), dtype=FP8, device=go.device)
        s = torch.empty((_blocks(K), M), dtype=_F32, device=go.device)
    _capi.moe_fp4_fp8_quantize(x.data_ptr(), row, act, q.data_ptr(), K, s.data_ptr(), 1, M, M, K, go.stream)
    return q, s.t()


def _product_operands(w, w_scale, addend, out, out_dtype, go, M, K):
    w_row = _matrix(w, "w", (FP8,), go.device, cols=K)
    N = w.shape[0]
    ws_row = _matrix(w_scale, "w_scale", (_F32,), go.device, _blocks(N), _blocks(K))
    add_row = 0 if addend is None else _matrix(addend, "addend", (_BF16,), go.device, M, N)
    if out is None:
        with go:
            out = torch.empty((M, N), dtype=out_dtype or _BF16, device=go.device)
        out_row = N
    else:
        out_row = _matrix(out, "out", (_BF16, _F32) if out_dtype is None else (out_dtype,), go.device, M, N)
    if out.dtype is not _BF16 and out.dtype is not _F32:
        raise TypeError(f"out must be bfloat16 or float32, not {out.dtype}")
    return (w.data_ptr(), w_row, w_scale.data_ptr(), ws_row, 0 if addend is None else addend.data_ptr(), add_row,
            out.data_ptr(), out_row, 1 if out.dtype is _F32 else 0, M, N, K), out


def fp8_matmul(x_q: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
               out: Optional[torch.Tensor] = None, addend: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """``out [M, N] = x @ w.T (+ addend)`` for E4M3 ``x_q [M, K]`` with scales
    ``x_scale [M, ceil(K / 128)]`` (any strides) and E4M3 ``w [N, K]`` with
    scales ``w_scale [ceil(N / 128), ceil(K / 128)]``; out bfloat16 (default)
    or float32, rounded once after the bfloat16 ``addend [M, N]``."""
    go = _Launch(x_q, stream)
    row = _matrix(x_q, "x_q", (FP8,), go.device)
    M, K = x_q.shape
    if x_scale.dtype is not _F32:
        raise TypeError(f"x_scale must be float32, not {x_scale.dtype}")
    if x_scale.shape != (M, _blocks(K)):
        raise ValueError(f"x_scale must be [{M}, {_blocks(K)}], not {list(x_scale.shape)}")
    if x_scale.device != go.device:
        raise ValueError(f"x_scale is on {x_scale.device}, not {go.device}")
    args, out = _product_operands(w, w_scale, addend, out, out_dtype, go, M, K)
    _capi.moe_fp4_fp8_matmul(x_q.data_ptr(), row, x_scale.data_ptr(), x_scale.stride(0), x_scale.stride(1), *args,
                             go.stream)
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
    to 16 rows of at most 16384 columns need none)."""
    go = _Launch(x, stream)
    row = _matrix(x, "x", (_BF16,), go.device)
    M, K = x.shape
    args, out = _product_operands(w, w_scale, addend, out, out_dtype, go, M, K)
    ws_ptr = ws_bytes = 0
    if workspace is None:
        if M > 16 or K > 16384:
            with go:
                workspace = torch.empty(_capi.moe_fp4_fp8_linear_workspace_bytes(M, K), dtype=torch.uint8,
                                        device=go.device)
    elif workspace.device != go.device or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on x's device")
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    _capi.moe_fp4_fp8_linear(x.data_ptr(), row, *args, ws_ptr, ws_bytes, go.stream)
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
    go = _Launch(residual, stream)
    dev = go.device
    a = _capi.MoeFp4BlockNormArgs()
    a.residual_row = _matrix(residual, "residual", (_BF16, _F32), dev)
    M, H = residual.shape
    a.M, a.H = M, H
    a.residual = residual.data_ptr()
    a.residual_f32 = 1 if residual.dtype is _F32 else 0
    a.scale, a.eps, a.offset = scale, eps, weight_offset
    wdt = (_BF16, _F32)
    for name, w in (("pre_weight", pre_weight), ("post_weight", post_weight)):
        if w is not None:
            _vector(w, name, wdt, dev, H)
            a.weights_f32 = 1 if w.dtype is _F32 else 0
            wdt = (w.dtype,)
    if block_out is None:
        if post_weight is not None or gate is not None:
            raise ValueError("post_weight and gate need block_out")
    else:
        a.block_row = _matrix(block_out, "block_out", (_BF16,), dev, M, H)
        a.block_out = block_out.data_ptr()
        if post_weight is not None:
            a.w_post = post_weight.data_ptr()
        if gate is not None:
            _gate(a, gate, dev, M, H)
    if pre_weight is None and (quantize or block_out is None):
        raise ValueError("without pre_weight there is nothing to " + ("quantize" if quantize else "compute"))
    normed = q = s = None
    with go:
        if residual_out is not None:
            a.residual_out_row = _matrix(residual_out, "residual_out", (residual.dtype,), dev, M, H)
            a.residual_out = residual_out.data_ptr()
        elif block_out is not None:
            residual_out = torch.empty((M, H), dtype=residual.dtype, device=dev)
            a.residual_out_row = H
            a.residual_out = residual_out.data_ptr()
        else:
            residual_out = residual
        if pre_weight is not None:
            a.w_pre = pre_weight.data_ptr()
            normed = torch.empty((M, H), dtype=_BF16, device=dev)
            a.normed, a.normed_row = normed.data_ptr(), H
        if quantize:
            q = torch.empty((M, H), dtype=FP8, device=dev)
            s = torch.empty((_blocks(H), M), dtype=_F32, device=dev)
            a.q, a.q_row, a.s, a.s_row, a.s_block = q.data_ptr(), H, s.data_ptr(), 1, M
    _capi.moe_fp4_block_norm(a, go.stream)
    return (residual_out, normed, q, s.t()) if quantize else (residual_out, normed)


def _gate(a, gate, dev, M, H):
    if gate.dtype not in (_BF16, _F32):
        raise TypeError(f"gate must be bfloat16 or float32, not {gate.dtype}")
    if gate.device != dev:
        raise ValueError(f"gate is on {gate.device}, not {dev}")
    if gate.shape == (H,):
        a.gate_row, a.gate_col = 0, gate.stride(0)
    elif gate.shape == (M, H):
        a.gate_row, a.gate_col = gate.stride()
    elif gate.shape == (M, 1):
        a.gate_row, a.gate_col = gate.stride(0), 0
    else:
        raise ValueError(f"gate must be [{H}], [{M}, 1] or [{M}, {H}], not {list(gate.shape)}")
    if a.gate_col not in (0, 1):
        raise ValueError("gate must have contiguous columns")
    a.gate, a.gate_f32 = gate.data_ptr(), 1 if gate.dtype is _F32 else 0


# ----------------------------------------------------------------------- router
def route_topk(logits: torch.Tensor, top_k: int, score: int = SCORE_SOFTMAX, bias: Optional[torch.Tensor] = None,
               renormalize: bool = True, scale: float = 1.0, stream=None):
    """``logits [M, E]`` (bfloat16 or float32) -> (``topk_ids`` int32
    ``[M, top_k]``, ``topk_weights`` float32 ``[M, top_k]``), as ``forward``
    takes them.  SCORE_SOFTMAX chooses by logit; SCORE_SIGMOID by
    sigmoid(logit) + ``bias`` (float32 ``[E]`` or None) and weighs by
    sigmoid(logit).  Equal scores go to the lowest index; experts with a logit
    of -inf or NaN are never chosen, and a row that runs out of experts ends
    in id -1 with weight 0.  ``renormalize`` divides by the chosen weights'
    sum; ``scale`` multiplies the weights."""
    go = _Launch(logits, stream)
    row = _matrix(logits, "logits", (_F32, _BF16), go.device)
    M, E = logits.shape
    if bias is not None:
        _vector(bias, "bias", (_F32,), go.device, E)
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    with go:
        ids = torch.empty((M, top_k), dtype=torch.int32, device=go.device)
        weights = torch.empty((M, top_k), dtype=_F32, device=go.device)
    _capi.moe_fp4_route_topk(logits.data_ptr(), row, 1 if logits.dtype is _F32 else 0,
                             None if bias is None else bias.data_ptr(), score, 1 if renormalize else 0, scale,
                             ids.data_ptr(), weights.data_ptr(), M, E, top_k, go.stream)
    return ids, weights
