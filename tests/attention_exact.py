"""The attention over a cache in 64 bits, with tables that may be shorter than
their requests, and how far the kernels may be from it."""
from __future__ import annotations

import math

import torch

from tests.attention_util import F64, Batch


def want(b: Batch, q, offsets, scale, window=0, sinks=None, k_scale=1.0, v_scale=1.0, capacity=None):
    """(out, lse, bound of out, bound of lse).

    A score x (in 64 bits) is off by 2^-18 of the sum of its terms'
    magnitudes (exact terms, FP32 sums of at most 256, three roundings), and a
    probability by d = that + 2^-21 (1 + |x| + |m|) of itself (the hardware's
    2^x and its argument, in units of log 2), then by 2^-11 of itself as FP16,
    or, below FP16's normal range, by 2^-25 in a measure in which the row's
    largest is at least 2^7: by 2^-32 of the largest, of which the divisor is
    no less.  FP32 sums add 2^-20, the output's rounding 2^-8."""
    T, Hq, D = q.shape
    G = Hq // b.Hkv
    out = torch.zeros(T, Hq, D, dtype=F64)
    lse = torch.full((T, Hq), -math.inf, dtype=F64)
    d_out, d_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for r, L in enumerate(b.lengths):
        lo, hi = offsets[r], min(offsets[r + 1], T)
        n = hi - lo
        if n <= 0:
            continue
        S = L if capacity is None else min(L, capacity)
        at = torch.arange(n)[:, None] + (L - n)
        j = torch.arange(S)
        sees = j <= at
        if window:
            sees &= j > at - window
        for h in range(Hq):
            qq = q[lo:hi, h].double()
            k, v = b.k[r][:S, h // G] * k_scale, b.v[r][:S, h // G] * v_scale
            x = (qq @ k.T * scale).masked_fill(~sees, -math.inf)
            sink = torch.full((n, 1), -math.inf if sinks is None else float(sinks[h]), dtype=F64)
            z = torch.logsumexp(torch.cat([x, sink], 1), 1)
            lse[lo:hi, h] = z
            finite = z.isfinite()
            z = torch.where(finite, z, 0.0)
            p = torch.exp(x - z[:, None])
            out[lo:hi, h] = p @ v
            if S:
                mag = (qq.abs() @ k.abs().T * abs(scale)).masked_fill(~sees, 0.0)
                d = (2.0 ** -18 * mag + 2.0 ** -21 * (1 + 2 * x.abs().masked_fill(~sees, 0.0))).amax(1, keepdim=True)
                d_out[lo:hi, h] = (p @ v.abs()) * (2 * d + 2.0 ** -11 + 2.0 ** -20) + 2.0 ** -32 * (sees.double() @ v.abs())
                d_lse[lo:hi, h] = d[:, 0] + 2.0 ** -20
            d_lse[lo:hi, h] += 2.0 ** -22 * z.abs()
    return out, lse, d_out + 2.0 ** -8 * (out.abs() + d_out), d_lse
