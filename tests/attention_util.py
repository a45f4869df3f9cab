"""Plain 64-bit forms of the operators on a paged cache of 4 bits, and caches
made on the host, for their tests."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64)


def e2m1_codes(x):
    """Codes 0 .. 7 of |x| to the nearest E2M1 value, ties to the even code."""
    half = (GRID[1:] + GRID[:-1]) / 2
    a = x.abs().double()
    up, down = torch.bucketize(a, half, right=True), torch.bucketize(a, half, right=False)
    return torch.where(up % 2 == 0, up, down)


def quantise(u):
    """[..., D] (taken to FP32) -> (codes [..., D] with the sign in bit 3, scales [..., D / 16] as E4M3)."""
    b = u.float().unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.double().unsqueeze(-1)
    code = torch.where(s > 0, e2m1_codes(b.double() / torch.where(s > 0, s, torch.ones_like(s))), 0)
    return (code + 8 * (torch.signbit(b) & (s > 0))).flatten(-2).to(torch.uint8), scale


def dequantise(code, scale):
    v = torch.where(code >= 8, -1.0, 1.0).double() * GRID[(code & 7).long()]
    return (v.unflatten(-1, (-1, 16)) * scale.double().unsqueeze(-1)).flatten(-2)


def store(cache, slot, head, kind, code, scale):
    """One token's codes [D] and scales [D / 16] into a cache (on the host)."""
    D = code.numel()
    page_size = cache.shape[2] * 16
    block = cache[slot // page_size, head, slot % page_size // 16, kind]
    row = slot % 16
    block[row * D // 2:(row + 1) * D // 2] = code[0::2] | (code[1::2] << 4)
    block[8 * D + row * D // 16:8 * D + (row + 1) * D // 16] = scale.view(torch.uint8)


def stored(cache, slots, D):
    """(k, v) [T, Hkv, D] in 64 bits of a cache on the host, without its FP32 scales."""
    page_size = cache.shape[2] * 16
    s = torch.as_tensor(slots)
    blocks = cache[s // page_size, :, s % page_size // 16]  # [T, Hkv, 2, 9 D]
    row = s % 16
    byte = blocks[..., :8 * D].unflatten(-1, (16, D // 2))[torch.arange(len(s)), :, :, row]
    scale = blocks[..., 8 * D:].unflatten(-1, (16, D // 16))[torch.arange(len(s)), :, :, row]
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    v = dequantise(code, scale.contiguous().view(torch.float8_e4m3fn))
    return v[:, :, 0], v[:, :, 1]


class Batch:
    """Requests with keys and values in a cache on the host; everything outside them is NaN scales."""

    def __init__(self, lengths, D, Hkv, page_size, seed=0, spare=3, k_std=1.0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page_size) for n in lengths]
        pages = sum(need) + spare
        self.D, self.Hkv, self.page_size, self.lengths = D, Hkv, page_size, lengths
        self.cache = torch.full((pages, Hkv, page_size // 16, 2, 9 * D), 0xff, dtype=torch.uint8)
        order = torch.randperm(pages, generator=g).tolist()
        width = max(need + [1]) + 1
        self.tables = torch.full((len(lengths), width), -1, dtype=torch.int32)
        self.k, self.v = [], []
        at = 0
        for r, n in enumerate(lengths):
            mine = order[at:at + need[r]]
            at += need[r]
            self.tables[r, :need[r]] = torch.tensor(mine, dtype=torch.int32)
            kc, ks = quantise(torch.randn(n, Hkv, D, generator=g) * k_std)
            vc, vs = quantise(torch.randn(n, Hkv, D, generator=g))
            self.k.append(dequantise(kc, ks))
            self.v.append(dequantise(vc, vs))
            for page in range(need[r]):
                lo, hi = page * page_size, min((page + 1) * page_size, n)
                for kind, (c, s) in enumerate(((kc, ks), (vc, vs))):
                    # [tokens, Hkv, ...] -> [Hkv, blocks, 16, ...]
                    full_c = torch.full((page_size, Hkv, D // 2), 0xff, dtype=torch.uint8)
                    full_s = torch.full((page_size, Hkv, D // 16), 0xff, dtype=torch.uint8)
                    full_c[:hi - lo] = c[lo:hi, :, 0::2] | (c[lo:hi, :, 1::2] << 4)
                    full_s[:hi - lo] = s[lo:hi].view(torch.uint8)
                    nb = page_size // 16
                    dst = self.cache[mine[page], :, :, kind]
                    dst[..., :8 * D] = full_c.view(nb, 16, Hkv, -1).permute(2, 0, 1, 3).reshape(Hkv, nb, -1)
                    dst[..., 8 * D:] = full_s.view(nb, 16, Hkv, -1).permute(2, 0, 1, 3).reshape(Hkv, nb, -1)

    def want(self, q, offsets, scale, window=0, sinks=None, k_scale=1.0, v_scale=1.0):
        """(out, lse, bound of out, bound of lse) in 64 bits.

        The products q . k are exact terms summed in FP32 by the matrix
        instructions: off by at most 2^-18 of the sum of their magnitudes (D
        <= 256 terms, each partial sum cut at 2^-23 of itself or rounded, and
        what is scaled afterwards rounded three times).  With the hardware's
        2^x (2 units, and half a unit of its argument, whose magnitude is at
        most that of x and of the maximum) a probability is off by d = 2^-18
        sum|q k| scale + 2^-21 (1 + |x| + |m|) of itself, then rounded to FP16
        (2^-11 of itself, or 2^-25 below FP16's normal range).  out moves by
        at most twice the largest d, and 2^-11, of the mean of |v|, and what
        the smallest leave; FP32 sums of n values add 2^-20; the output is
        rounded to BF16 (2^-8)."""
        T, Hq, D = q.shape
        G = Hq // self.Hkv
        out = torch.zeros(T, Hq, D, dtype=F64)
        lse = torch.full((T, Hq), -math.inf, dtype=F64)
        d_out, d_lse = torch.zeros_like(out), torch.zeros_like(lse)
        for r, L in enumerate(self.lengths):
            lo, hi = offsets[r], min(offsets[r + 1], T)
            n = hi - lo
            if n <= 0:
                continue
            at = torch.arange(n)[:, None] + (L - n)
            j = torch.arange(L)
            sees = j <= at
            if window:
                sees &= j > at - window
            for h in range(Hq):
                qq = q[lo:hi, h].double()
                k, v = self.k[r][:, h // G] * k_scale, self.v[r][:, h // G] * v_scale
                x = torch.where(sees, qq @ k.T * scale, torch.tensor(-math.inf, dtype=F64))
                mag = (qq.abs() @ k.abs().T) * abs(scale)
                if sinks is not None:
                    sink = sinks[h].double().expand(n, 1)
                    lse[lo:hi, h] = torch.logsumexp(torch.cat([x, sink], 1), 1)
                else:
                    lse[lo:hi, h] = torch.logsumexp(x, 1) if L else -math.inf
                z = lse[lo:hi, h, None]
                p = torch.where(sees, torch.exp(x - z), torch.zeros_like(x)) if L else torch.zeros(n, 0, dtype=F64)
                out[lo:hi, h] = p @ v
                if L:
                    xs = torch.where(sees, x.abs(), torch.zeros_like(x))
                    d = (2.0 ** -18 * torch.where(sees, mag, torch.zeros_like(mag)) + 2.0 ** -21 * (1 + 2 * xs)).amax(1, keepdim=True)
                    # (FP16's values below 2^-14 lie 2^-24 apart: a probability there, taken against the row's
                    # largest of 1, is off by 2^-25, and the divisor is at least 1 in the same measure, so that
                    # out moves by 2^-25 of the sum of |v|)
                    d_out[lo:hi, h] = p @ v.abs() * (2 * d + 2.0 ** -11 + 2.0 ** -20) + 2.0 ** -25 * sees.double() @ v.abs()
                    d_lse[lo:hi, h] = (d + 2.0 ** -20)[:, 0]
                # (to units of log 2 and back: two products, two rounded factors)
                d_lse[lo:hi, h] += 2.0 ** -22 * torch.where(z[:, 0].isfinite(), z[:, 0].abs(), torch.zeros_like(z[:, 0]))
        d_out = d_out + 2.0 ** -8 * (out.abs() + d_out)
        return out, lse, d_out, d_lse


def check(got, want, bound, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    err = (got - want).abs()
    worst = float((err / bound.clamp(min=1e-30)).max()) if err.numel() else 0.0
    assert (err <= bound).all(), (what, worst)


def check_lse(got, want, bound, what=""):
    got = got.double().cpu()
    assert torch.equal(got == -math.inf, want == -math.inf), what
    fine = want != -math.inf
    err = (got - want).abs()[fine]
    assert (err <= bound[fine]).all(), (what, float((err / bound[fine].clamp(min=1e-30)).max()))
