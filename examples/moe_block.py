#!/usr/bin/env python3
"""One mixture-of-experts block of a decoder, as a serving loop runs it:

    r, n, q, s   = block_norm(r, w_pre, b, post_weight=w_post, quantize=True)   previous block's end, this one's start
    ids, weights = route_topk(n @ w_router.T, top_k)                            the router's choice
    y            = forward(n, experts, ids, weights)                            routed FP4 experts
    q, s         = fp8_quantize(fp8_matmul(q, s, w_gate_up), act=ACT_SILU)      the shared expert, always on, in FP8
    b            = fp8_matmul(q, s, w_down, addend=y)                           ... its output added to the routed sum

and the next block's block_norm takes (r, b) on.  Weights and activations are
random.  The block runs eagerly and from a CUDA graph, is compared with a
plain FP32 computation on the dequantised weights, and is timed.

    python examples/moe_block.py [--tokens 4] [--experts 64] [--hidden 2560] [--intermediate 320] [--top-k 10]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fp4_weight_moe_gb300 as m  # noqa: E402
from workload import gen  # noqa: E402


def fp8_weight(rows: int, cols: int, g: torch.Generator):
    """A random FP8 checkpoint weight: E4M3 values, an FP32 scale per 128 x 128 block."""
    w = torch.randn(rows, cols, generator=g, device="cuda") * 0.02
    nr, nc = -(-rows // 128), -(-cols // 128)
    tiles = torch.nn.functional.pad(w, (0, nc * 128 - cols, 0, nr * 128 - rows)).view(nr, 128, nc, 128)
    s = tiles.abs().amax(dim=(1, 3)) / 448.0
    q = (tiles / s[:, None, :, None]).reshape(nr * 128, nc * 128)[:rows, :cols]
    return q.contiguous().to(torch.float8_e4m3fn), s


class MoEBlock:
    """Weights and scratch of one block for up to ``max_tokens`` tokens."""

    def __init__(self, E: int, H: int, I: int, top_k: int, max_tokens: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.top_k = top_k
        self.logical = gen.make_expert_weights(E, H, I, gen.NVFP4, seed, device="cuda")
        self.experts = m.prepare_weights(self.logical, E, H, I, m.NVFP4)
        self.workspace = m.alloc_workspace(max_tokens, E, H, I, top_k, m.NVFP4)
        self.router = (torch.randn(E, H, generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)
        self.gate_up, self.gate_up_scale = fp8_weight(2 * I, H, g)
        self.down, self.down_scale = fp8_weight(H, I, g)
        self.w_pre = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        self.w_post = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)

    def __call__(self, residual: torch.Tensor, block_out: torch.Tensor):
        """(residual stream, previous block's output) -> (residual stream, this block's output)."""
        residual, n, q, s = m.block_norm(residual, self.w_pre, block_out, post_weight=self.w_post, quantize=True)
        ids, weights = m.route_topk(n @ self.router.t(), self.top_k)
        routed = m.forward(n, self.experts, ids, weights, workspace=self.workspace)
        gate_up = m.fp8_matmul(q, s, self.gate_up, self.gate_up_scale)
        q, s = m.fp8_quantize(gate_up, act=m.ACT_SILU)
        return residual, m.fp8_matmul(q, s, self.down, self.down_scale, addend=routed)

    # ------------------------------------------------------------ plain FP32 form
    def plain(self, residual: torch.Tensor, block_out: torch.Tensor):
        def rms(v, w):
            return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w.float()

        def dense(q, s):
            r, c = q.shape
            return q.float() * s.repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :c]

        r = residual.float() + rms(block_out.float(), self.w_post)
        n = rms(r, self.w_pre).to(torch.bfloat16)
        logits = (n @ self.router.t()).float()
        top, ids = torch.topk(logits, self.top_k, dim=1)
        weights = torch.softmax(top, dim=1)
        x = n.float()
        out = torch.zeros_like(x)
        I = self.experts.I
        for t in range(x.shape[0]):
            for e, w in zip(ids[t].tolist(), weights[t].tolist()):
                w13, w2 = m.debug_dequant(self.experts, 0, e), m.debug_dequant(self.experts, 1, e)
                h = w13 @ x[t]
                out[t] += w * (w2 @ (torch.nn.functional.silu(h[:I]) * h[I:]))
        h = x @ dense(self.gate_up, self.gate_up_scale).t()
        shared = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ dense(self.down, self.down_scale).t()
        return r, out + shared


def cosine(a: torch.Tensor, b: torch.Tensor) -> float:
    return float(torch.nn.functional.cosine_similarity(a.double().flatten(), b.double().flatten(), dim=0))


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--intermediate", type=int, default=320)
    ap.add_argument("--top-k", type=int, default=10)
    a = ap.parse_args(argv)
    block = MoEBlock(a.experts, a.hidden, a.intermediate, a.top_k, a.tokens)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    residual = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    previous = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)

    r, b = block(residual, previous)
    want_r, want_b = block.plain(residual, previous)
    result = dict(cos_residual=cosine(r, want_r), cos_block=cosine(b, want_b))

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        block(residual, previous)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            graph_r, graph_b = block(residual, previous)
        graph.replay()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record(stream)
        for _ in range(20):
            graph.replay()
        end.record(stream)
        stream.synchronize()
    result["us_per_block"] = start.elapsed_time(end) / 20 * 1e3
    result["cos_graph"] = cosine(graph_b, b)
    assert m.workspace_status(block.workspace) == 0 and m.fp8_status() == 0
    print(" ".join(f"{k}={v:.6g}" for k, v in result.items()))
    return result


if __name__ == "__main__":
    main()
