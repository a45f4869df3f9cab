"""The cache's operators together, as a serving loop runs them: pages and slots
for a step's tokens, the store of keys and values, attention over the cache;
prompts, chunks and decoding, requests that end and rows that are used anew;
eagerly against 64 bits, and from a CUDA graph against the eager run."""
import math

import pytest
import torch

from tests.attention_util import Batch, check, dequantise, quantise
from tests.gpu_util import ensure_built
from tests.test_qk_norm_rope_gpu import formula

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


class Server:
    """What a serving loop keeps for one layer."""

    def __init__(self, m, R, Hq, Hkv, D, page, pages, width):
        self.m, self.R, self.Hq, self.Hkv, self.D, self.page = m, R, Hq, Hkv, D, page
        self.cache = m.alloc_fp4_cache(pages, page, Hkv, D)
        self.tables = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(0)).to(torch.int32).cuda()
        self.count = torch.tensor([pages], dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.rotary = m.rotary_table(4096, D // 2)
        g = torch.Generator().manual_seed(1)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(BF16).cuda() for _ in range(2))
        self.workspace = m.alloc_fp4_attention_workspace(R, Hq, Hkv, D)

    def step(self, qkv, new, ends=None):
        m, Hq, Hkv, D = self.m, self.Hq, self.Hkv, self.D
        T = qkv.shape[0]
        st = m.cache_step(self.lengths, new, self.tables, self.free, self.count, self.page, T, finished=ends,
                          lengths_out=self.lengths, free_count_out=self.count)
        x = qkv.view(T, Hq + 2 * Hkv, D)
        q, _ = m.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], st.positions, self.rotary, q_weight=self.wq,
                              k_weight=self.wk, v=x[:, Hq + Hkv:], cache=self.cache, slots=st.slots, k_scale=0.5,
                              v_scale=0.8)
        out = m.fp4_attention(q, self.cache, self.tables, self.lengths, st.offsets, k_scale=0.5, v_scale=0.8,
                              workspace=self.workspace)
        return out, q, st


class Model:
    """The same in 64 bits, request by request, from q as it was rounded to BF16."""

    def __init__(self, s: Server):
        self.s, self.k, self.v = s, [[] for _ in range(s.R)], [[] for _ in range(s.R)]

    def step(self, qkv, q, new, ends=None):
        s, at = self.s, 0
        x = qkv.cpu().view(-1, s.Hq + 2 * s.Hkv, s.D)
        lengths = []
        for r, n in enumerate(new):
            if ends is not None and ends[r]:
                self.k[r], self.v[r] = [], []
            for i in range(n):
                table = s.rotary.cpu()[len(self.k[r])][None]
                k = formula(x[at + i, None, s.Hq:s.Hq + s.Hkv], s.wk.cpu(), table, float(torch.tensor(1e-6)), 0.0, False)[0]
                self.k[r].append(dequantise(*quantise(k[0].float() / 0.5)))
                self.v[r].append(dequantise(*quantise(x[at + i, s.Hq + s.Hkv:].float() / torch.tensor(0.8))))
            lengths.append(len(self.k[r]))
            at += n
        b = Batch.__new__(Batch)
        b.D, b.Hkv, b.lengths = s.D, s.Hkv, lengths
        empty = torch.zeros(0, s.Hkv, s.D, dtype=torch.float64)
        b.k = [torch.stack(k) if k else empty for k in self.k]
        b.v = [torch.stack(v) if v else empty for v in self.v]
        offsets = [0]
        for n in new:
            offsets.append(offsets[-1] + n)
        return b.want(q.cpu(), offsets, 1 / math.sqrt(s.D), 0, None, 0.5, 0.8)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 16), (6, 6, 64, 32), (10, 2, 256, 64)])
def test_serving_loop(Hq, Hkv, D, page):
    m = _m()
    s = Server(m, 4, Hq, Hkv, D, page, 48, 24 * 16 // page + 1)
    model = Model(s)
    g = torch.Generator().manual_seed(5)
    steps = [([70, 1, 0, 33], None), ([1, 1, 40, 1], None), ([1, 1, 1, 1], None), ([1, 0, 1, 50], [0, 0, 0, 1]),
             ([30, 1, 1, 1], [0, 1, 0, 0]), ([1, 1, 1, 1], None)]
    for new, ends in steps:
        pad = 3
        qkv = torch.randn(sum(new) + pad, (Hq + 2 * Hkv) * D, generator=g).to(BF16).cuda()
        mask = None if ends is None else torch.tensor(ends, dtype=torch.bool, device="cuda")
        out, q, st = s.step(qkv, ints(new), mask)
        assert st.accepted.tolist() == new
        want = model.step(qkv[:sum(new)], q, new, ends)
        check(out[:sum(new)], want[0][:sum(new)], want[2][:sum(new)], (new, ends))
        assert (out[sum(new):] == 0).all()
    assert s.lengths.tolist() == [len(k) for k in model.k]
    used = sum(-(-n // page) for n in s.lengths.tolist())
    assert int(s.count) == 48 - used
    held = [int(s.tables[r, j]) for r in range(4) for j in range(-(-int(s.lengths[r]) // page))]
    assert sorted(held + s.free[:48 - used].tolist()) == list(range(48))
    assert m.fp4_attention_status() == 0


@pytest.mark.parametrize("new", [1, 20])
def test_captured_step(new):
    """A step captured once and replayed, its lengths and pages carried on in place."""
    m = _m()
    R, Hq, Hkv, D = 3, 8, 2, 128
    eager, captured = (Server(m, R, Hq, Hkv, D, 16, 60, 20) for _ in range(2))
    g = torch.Generator().manual_seed(2)
    first = torch.randn(90, (Hq + 2 * Hkv) * D, generator=g).to(BF16).cuda()
    for s in (eager, captured):
        s.step(first, ints([60, 1, 29]))
    qkv, count = first[:R * new].clone(), ints([new] * R)
    state = [t.clone() for t in (captured.cache, captured.tables, captured.free, captured.count, captured.lengths)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        captured.step(qkv, count)
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out, q, st = captured.step(qkv, count)
    torch.cuda.synchronize()
    for t, v in zip((captured.cache, captured.tables, captured.free, captured.count, captured.lengths), state):
        t.copy_(v)
    for i in range(6):
        x = torch.randn(R * new, (Hq + 2 * Hkv) * D, generator=g).to(BF16).cuda()
        qkv.copy_(x)
        graph.replay()
        want, _, st2 = eager.step(x, count)
        assert torch.equal(out, want) and torch.equal(st.slots, st2.slots), i
    assert torch.equal(captured.lengths, eager.lengths) and torch.equal(captured.cache, eager.cache)


def test_two_streams_at_once():
    """Calls on two streams, each with its own scratch, give what they give alone."""
    m = _m()
    cases = []
    for seed, (lengths, new) in enumerate((([3000, 50, 700], [1, 1, 1]), ([400, 900], [60, 130]))):
        b = Batch(lengths, 128, 2, 32, seed)
        q = torch.randn(sum(new), 8, 128, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        args = (q, b.cache.cuda(), b.tables.cuda(), ints(lengths), ints(off))
        cases.append((args, m.fp4_attention(*args)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (args, _) in enumerate(cases):
            got[i].append(m.fp4_attention(*args, stream=streams[i]))
    torch.cuda.synchronize()
    for i, (_, want) in enumerate(cases):
        assert all(torch.equal(o, want) for o in got[i])
