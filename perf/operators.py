"""Performance cases of the operators around the MoE layer: the FP8 product
with a scale per block of 128, the norms before and after a block with its
gate and residual scale, and the router's choice of experts.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, by the calls a
user makes of the package.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the shared expert's gate-and-up projection: weights streamed once
        dict(name="fp8_decode", op="linear", M=1, K=7168, N=4096, out="bf16"),
        # a serving batch's down projection: gated activation, quantisation, product added to the routed experts' sum
        dict(name="fp8_gated_down", op="gated", M=64, K=2048, N=7168, out="bf16"),
        # a long prompt through a wide projection: tensor-core bound
        dict(name="fp8_prefill", op="linear", M=4096, K=7168, N=4096, out="bf16"),
        # sizes that fill no tile, FP32 output (a router projection)
        dict(name="fp8_ragged", op="linear", M=333, K=2576, N=1000, out="f32"),
        # one token between two blocks: latency
        dict(name="norm_decode", op="norm", M=1, H=2560, res="bf16", gate="none", post=True),
        # a serving batch, FP32 residual stream, a learned gate per channel
        dict(name="norm_batch", op="norm", M=64, H=7168, res="f32", gate="channel", post=True),
        # a prompt with the sandwich norms
        dict(name="norm_prefill", op="norm", M=4096, H=4096, res="bf16", gate="none", post=True),
        # a long prompt with a gate for each token and no norm after the block
        dict(name="norm_long", op="norm", M=16384, H=7168, res="bf16", gate="token", post=False),
        # a width that no vector load divides, gate for each element
        dict(name="norm_odd", op="norm", M=777, H=1283, res="f32", gate="full", post=True),
        # norm, quantisation and the shared expert's first projection, as a decode step runs them
        dict(name="norm_fp8", op="norm_linear", M=8, H=4096, N=1024, res="bf16"),
        # router of a few decoding tokens, softmax scores
        dict(name="router_decode", op="router", M=4, E=288, k=10, score="softmax", logits="f32", masked=2),
        # router of a prompt, sigmoid scores with a correction bias
        dict(name="router_prefill", op="router", M=4096, E=512, k=10, score="sigmoid", logits="f32", masked=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "gated", "norm", "norm", "norm_linear", "router"])
    if op in ("linear", "gated"):
        K = 16 * _log(rng, 16, 448)  # 256 .. 7168
        N = _log(rng, 200, 7168)
        M = _log(rng, 1, 4096)
        while M * N * K > 4096 * 7168 * 4096:
            M = max(1, M // 2)
        return dict(op=op, M=M, K=K, N=N, out=rng.choice(["bf16", "bf16", "f32"]) if op == "linear" else "bf16")
    if op == "norm":
        H = _log(rng, 200, 8192)
        if rng.random() < 0.6:
            H = max(256, H // 64 * 64)
        M = _log(rng, 1, 16384)
        while M * H > 16384 * 4096:
            M //= 2
        return dict(op=op, M=M, H=H, res=rng.choice(["bf16", "f32"]),
                    gate=rng.choice(["none", "channel", "token", "full"]), post=rng.random() < 0.7)
    if op == "norm_linear":
        return dict(op=op, M=_log(rng, 1, 512), H=256 * _log(rng, 1, 28), N=_log(rng, 200, 4096),
                    res=rng.choice(["bf16", "f32"]))
    E = _log(rng, 8, 1024)
    return dict(op=op, M=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(16, E)),
                score=rng.choice(["softmax", "sigmoid"]), logits=rng.choice(["f32", "bf16"]), masked=rng.choice([0, E // 4]))


# --------------------------------------------------------------------- inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _weight(N, K, g):
    """A checkpoint's FP8 weight: N(0, 0.02) values, a scale per 128 x 128 block."""
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    pad = torch.nn.functional.pad(w, (0, _blocks(K) * BLOCK - K, 0, _blocks(N) * BLOCK - N))
    tiles = pad.view(_blocks(N), BLOCK, _blocks(K), BLOCK)
    s = tiles.abs().amax(dim=(1, 3)) / E4M3_MAX
    q = (tiles / s[:, None, :, None]).reshape(pad.shape)[:N, :K]
    return q.contiguous().to(torch.float8_e4m3fn), s.contiguous()


def _activation(M, K, g):
    """Unit-variance activations with a few strong channels."""
    x = torch.randn(M, K, generator=g, device="cuda")
    strong = torch.rand(K, generator=g, device="cuda") < 0.005
    return torch.where(strong, 20.0 * x, x).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("linear", "gated"):
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = _activation(M, K if op == "linear" else 2 * K, g)
        s["w"], s["ws"] = _weight(N, K, g)
        if op == "gated":
            s["add"] = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    elif op in ("norm", "norm_linear"):
        M, H = case["M"], case["H"]
        s["b"] = (torch.randn(M, H, generator=g, device="cuda") * 0.3).to(torch.bfloat16)
        s["r"] = (torch.randn(M, H, generator=g, device="cuda") * 2.0).to(_dtype(case["res"]))
        s["w_pre"] = (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s["w_post"] = (0.5 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s["w_post"] = s["w_post"] if case.get("post", True) else None
        s["scale"] = 0.7
        shape = {"none": None, "channel": (H,), "token": (M, 1), "full": (M, H)}[case.get("gate", "none")]
        s["g"] = None if shape is None else torch.rand(shape, generator=g, device="cuda").to(torch.bfloat16)
        if op == "norm_linear":
            s["w"], s["ws"] = _weight(case["N"], H, g)
    else:
        M, E = case["M"], case["E"]
        s["l"] = (torch.randn(M, E, generator=g, device="cuda") * 2.0).to(_dtype(case["logits"]))
        if case["masked"]:  # experts that a token may not take
            gone = torch.rand(M, E, generator=g, device="cuda").argsort(dim=1)[:, :case["masked"]]
            s["l"].scatter_(1, gone, float("-inf"))
        s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if case["score"] == "sigmoid" else None
    return s


# ---------------------------------------------------------------- plain forms
def _quantised(x):
    """x (32 bits) as the values its FP8 form stands for: a scale per row and 128 columns."""
    M, K = x.shape
    xb = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(M, _blocks(K), BLOCK)
    s = xb.abs().amax(dim=2, keepdim=True)
    s = s / torch.full_like(s, E4M3_MAX)  # a true division: by a Python number it would be a product with 1 / 448
    s = torch.where(s == 0, torch.ones_like(s), s)
    return ((xb / s).to(torch.float8_e4m3fn).float() * s).reshape(M, -1)[:, :K]


def _product(x, w, ws):
    N, K = w.shape
    s = ws.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return _quantised(x) @ (w.float() * s).t()


def _norm_of(v, w):
    return v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * w


def _norms(st):
    z = st["b"].float()
    if st["w_post"] is not None:
        z = _norm_of(z, st["w_post"].float())
    if st["g"] is not None:
        z = z * st["g"].float()
    r = st["r"].float() + st["scale"] * z
    return r, _norm_of(r, st["w_pre"].float())


def _router(st):
    logits = st["l"].float()
    fine = logits > float("-inf")
    order = logits if st["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-logits)) + st["bias"]
    order = torch.where(fine, order, torch.full_like(order, float("-inf")))
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :st["k"]]
    taken = torch.gather(fine, 1, ids)
    chosen = torch.gather(logits, 1, ids)
    if st["score"] == "softmax":
        v = torch.exp(chosen - chosen[:, :1])
    else:
        v = 1.0 / (1.0 + torch.exp(-chosen))
    v = torch.where(taken, v, torch.zeros_like(v))
    total = v.sum(dim=1, keepdim=True)
    weights = torch.where(total > 0, v / total, torch.zeros_like(v))
    return torch.where(taken, ids, torch.full_like(ids, -1)).int(), weights


def run(state):
    op = state["op"]
    if own:
        return _own(state)
    if op == "linear":
        return _product(state["x"].float(), state["w"], state["ws"]).to(_dtype(state["out"]))
    if op == "gated":
        gate, up = state["x"].float().chunk(2, dim=1)
        y = _product(gate / (1.0 + torch.exp(-gate)) * up, state["w"], state["ws"])
        return (y + state["add"].float()).to(torch.bfloat16)
    if op in ("norm", "norm_linear"):
        r, n = _norms(state)
        r, n = r.to(state["r"].dtype), n.to(torch.bfloat16)
        if op == "norm":
            return r, n
        return r, n, _product(n.float(), state["w"], state["ws"]).to(torch.bfloat16)
    return _router(state)


# ------------------------------------------------------------ the package's calls
def _own(st):
    import fp4_weight_moe_gb300 as m
    op = st["op"]
    if op == "linear":
        return m.fp8_linear(st["x"], st["w"], st["ws"], out_dtype=_dtype(st["out"]))
    if op == "gated":
        q, s = m.fp8_quantize(st["x"], act=m.ACT_SILU)
        return m.fp8_matmul(q, s, st["w"], st["ws"], addend=st["add"])
    if op == "norm":
        return m.block_norm(st["r"], st["w_pre"], st["b"], post_weight=st["w_post"], gate=st["g"], scale=st["scale"],
                            eps=EPS)
    if op == "norm_linear":
        r, n, q, s = m.block_norm(st["r"], st["w_pre"], st["b"], post_weight=st["w_post"], scale=st["scale"], eps=EPS,
                                  quantize=True)
        return r, n, m.fp8_matmul(q, s, st["w"], st["ws"])
    return m.route_topk(st["l"], st["k"], score=m.SCORE_SOFTMAX if st["score"] == "softmax" else m.SCORE_SIGMOID,
                        bias=st["bias"])


# ----------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("linear", "gated"):
        M, K, N = case["M"], case["K"], case["N"]
        moved = N * K + 4 * _blocks(N) * _blocks(K) + M * N * (2 if case["out"] == "bf16" else 4)
        moved += 2 * M * K if op == "linear" else 4 * M * K + 2 * M * N
        return dict(bytes=moved, flops=2 * M * N * K)
    if op in ("norm", "norm_linear"):
        M, H = case["M"], case["H"]
        res = 2 if case["res"] == "bf16" else 4
        gate = {"none": 0, "channel": 2 * H, "token": 2 * M, "full": 2 * M * H}[case.get("gate", "none")]
        moved = M * H * (2 + 2 * res + 2) + gate + 2 * H * (2 if case.get("post", True) else 1)
        flops = 10 * M * H
        if op == "norm_linear":
            N = case["N"]
            moved += N * H + 4 * _blocks(N) * _blocks(H) + 2 * M * N
            flops += 2 * M * N * H
        return dict(bytes=moved, flops=flops)
    M, E, k = case["M"], case["E"], case["k"]
    moved = M * E * (4 if case["logits"] == "f32" else 2) + 8 * M * k + (4 * E if case["score"] == "sigmoid" else 0)
    return dict(bytes=moved, flops=M * E * 2)


# ---------------------------------------------------------------------- exact
def _e4m3_64(v):
    """Nearest E4M3 value (ties to even) of |v| <= 448, in 64 bits."""
    m, _ = torch.frexp(v)  # |m| in [1/2, 1): four bits of it stay
    normal = torch.round(m * 16) / 16 * (v / torch.where(m == 0, torch.ones_like(m), m))
    return torch.where(v.abs() < 2.0 ** -6, torch.round(v * 512) / 512, normal)


def _linear_64(x, st):
    w, ws = st["w"].double(), st["ws"].double()
    N, K = w.shape
    n, k = torch.arange(N, device=w.device) // BLOCK, torch.arange(K, device=w.device) // BLOCK
    amax = torch.zeros(x.shape[0], _blocks(K), dtype=torch.float64, device=w.device)
    amax.scatter_reduce_(1, k.expand(x.shape[0], K), x.abs(), "amax")
    s = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))[:, k]
    return (_e4m3_64(x / s) * s) @ (w * ws[n][:, k]).t()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _linear_64(st["x"].double(), st)
    if op == "gated":
        K = case["K"]
        gate, up = st["x"][:, :K].double(), st["x"][:, K:].double()
        return _linear_64(gate * torch.sigmoid(gate) * up, st) + st["add"].double()
    if op in ("norm", "norm_linear"):
        z = st["b"].double()
        if st["w_post"] is not None:
            z = z / (z.pow(2).mean(1, keepdim=True) + EPS).sqrt() * st["w_post"].double()
        r = st["r"].double() + st["scale"] * (z if st["g"] is None else st["g"].double() * z)
        n = r / (r.pow(2).mean(1, keepdim=True) + EPS).sqrt() * st["w_pre"].double()
        return (r, n) if op == "norm" else (r, n, _linear_64(n.to(torch.bfloat16).double(), st))
    v = st["l"].double()
    order = v if case["score"] == "softmax" else torch.where(v > float("-inf"), v.sigmoid() + st["bias"].double(), v)
    ids = order.argsort(dim=1, descending=True, stable=True)[:, :case["k"]]
    v = v.gather(1, ids)
    if case["score"] == "softmax":
        return None, v.softmax(dim=1)
    v = v.sigmoid()
    return None, v / v.sum(dim=1, keepdim=True)
