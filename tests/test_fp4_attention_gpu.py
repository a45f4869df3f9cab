"""Attention over the cache of 4 bits against the formula in 64 bits (bounds:
attention_util.Batch.want)."""
import math

import pytest
import torch

from tests.attention_util import Batch, check, check_lse, stored
from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def sums(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def queries(T, Hq, D, seed, std=1.5):
    return (torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(seed)) * std).to(BF16)


def run(m, b, q, new, **kw):
    got = m.fp4_attention(q.cuda(), b.cache.cuda(), b.tables.cuda(), ints(b.lengths), ints(sums(new)), **kw)
    assert m.fp4_attention_status() == 0
    return got


def compare(lengths, new, D, Hq, Hkv, page, window=0, sinks=False, k_scale=1.0, v_scale=1.0, scale=None, seed=0, tail=0,
            k_std=1.0):
    m = _m()
    b = Batch(lengths, D, Hkv, page, seed, k_std=k_std)
    q = queries(sum(new) + tail, Hq, D, seed + 1)
    s = torch.randn(Hq, generator=torch.Generator().manual_seed(seed + 2)) if sinks else None
    out, lse = run(m, b, q, new, window=window, sinks=None if s is None else s.cuda(), k_scale=k_scale, v_scale=v_scale,
                   scale=scale, return_lse=True)
    want = b.want(q, sums(new), 1 / math.sqrt(D) if scale is None else scale, window, s, k_scale, v_scale)
    check(out, want[0], want[2])
    check_lse(lse, want[1], want[3])
    return out, lse


DIMS = [64, 128, 256]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("group", [1, 2, 5, 8, 9, 16, 17, 64])
def test_groups(D, group):
    compare([1, 15, 16, 17, 63, 64, 65, 200], [1] * 8, D, group, 1, 16)
    compare([77, 130], [1, 1], D, 2 * group, 2, 32, window=50, sinks=True, k_scale=0.5, v_scale=3.0)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pages(D, page):
    compare([page - 1, page, page + 1, 5 * page + 7], [1, 1, 1, 1], D, 8, 2, page, seed=page)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("window", [1, 15, 16, 17, 64, 300, 2 ** 31 - 1])
def test_windows(D, window):
    compare([1, 40, 300, 1000], [1, 3, 20, 2], D, 6, 2, 32, window=window, sinks=window == 17, seed=window % 100)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("sinks", [False, True])
def test_no_keys_and_no_queries(D, sinks):
    """Requests without tokens or without queries, queries before the first key, rows behind the last sequence."""
    lengths, new = [0, 3, 7, 0, 2, 33], [2, 0, 7, 0, 5, 1]
    out, lse = compare(lengths, new, D, 4, 2, 16, sinks=sinks, tail=4)
    off = sums(new)
    for rows in (out[0:2], out[off[4]:off[4] + 3], out[off[6]:]):
        assert (rows == 0).all()
    assert (lse[off[6]:] == -math.inf).all()


@pytest.mark.parametrize("new", [[9, 30], [60, 40], [400, 300]])
def test_widest_window_behind_queries_without_keys(new):
    """The first query's position less the window passes 32 bits; the window leaves out no key."""
    m = _m()
    b = Batch([3, 25], 128, 2, 16, 5)
    q = queries(sum(new), 4, 128, 6)
    want = run(m, b, q, new)
    got = run(m, b, q, new, window=2 ** 31 - 1, out=torch.full_like(want, 7.0))
    assert torch.equal(got, want)
    assert (want[new[0] - 1] != 0).any() and (want[-1] != 0).any()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("new", [[1, 2], [9, 12], [25, 31], [150, 90]])
def test_growing_scores(D, new):
    """Each 32 tokens' keys twice as large, so that the running maximum moves in most steps, and not in all rows."""
    m = _m()
    b = Batch([900, 333], D, 2, 64, 11)
    # (a scale's exponent, four bits above three of its fraction, up by one per 32 tokens, from 2^-6 on)
    for r, length in enumerate(b.lengths):
        for at in range(0, length, 16):
            scales = b.cache[int(b.tables[r, at // 64]), :, at % 64 // 16, 0, 8 * D:]
            larger = (scales & 7) | (min(1 + at // 32, 14) << 3)
            scales.copy_(torch.where((scales & 0x7f) == 0x7f, scales, larger))
        t = torch.arange(length)
        b.k[r] = stored(b.cache, b.tables[r, t // 64].long() * 64 + t % 64, D)[0]
    q = queries(sum(new), 8, D, 12)
    out, lse = run(m, b, q, new, return_lse=True)
    want = b.want(q, sums(new), 1 / math.sqrt(D), 0, None, 1.0, 1.0)
    check(out, want[0], want[2])
    check_lse(lse, want[1], want[3])


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("new", [[5] * 16, [8, 3, 6, 7] * 4, [31] * 16])
def test_many_items_to_a_worker_again_and_again(D, new):
    """Every item's end is waited for, however late a warp comes to it: no wait gives up in many calls."""
    m = _m()
    b = Batch([1500 + 37 * i for i in range(16)], D, 2, 32, 13)
    q = queries(sum(new), 8, D, 14)
    args = (q.cuda(), b.cache.cuda(), b.tables.cuda(), ints(b.lengths), ints(sums(new)))
    outs = [m.fp4_attention(*args) for _ in range(60)]
    assert m.fp4_attention_status() == 0
    want = b.want(q, sums(new), 1 / math.sqrt(D), 0, None, 1.0, 1.0)
    check(outs[0], want[0], want[2])
    for out in outs[1:]:
        assert torch.equal(out, outs[0])


def test_empty_batches():
    m = _m()
    cache = m.alloc_fp4_cache(2, 16, 2, 64)
    q = torch.ones(3, 4, 64, dtype=BF16, device="cuda")
    none = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    out, lse = m.fp4_attention(q, cache, none, none[:, 0], ints([0]), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert m.fp4_attention(q[:0], cache, none, none[:, 0], ints([0])).shape == (0, 4, 64)
    # tables without a column: no tokens to look for
    out = m.fp4_attention(q, cache, torch.zeros(1, 0, dtype=torch.int32, device="cuda"), ints([5]), ints([0, 3]))
    assert (out == 0).all()


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("new", [[2, 3, 5], [40, 1, 130], [300, 17, 1]])
@pytest.mark.parametrize("group", [1, 4, 7])
def test_chunks(D, new, group):
    compare([400, 257, 130], new, D, 2 * group, 2, 16, seed=group)
    compare(new, new, D, group, 1, 64, window=33, seed=group)


@pytest.mark.parametrize("D", DIMS)
def test_long(D):
    """One request over many workers, and many short ones."""
    compare([20000], [1], D, 4, 1, 128, seed=1)
    compare([9000, 1, 30], [2, 1, 1], D, 8, 1, 64, window=5000, seed=2)


@pytest.mark.parametrize("R", [100, 700])
def test_many_requests(R):
    lengths = [(37 * i) % 90 for i in range(R)]
    compare(lengths, [1 if i % 5 else 0 for i in range(R)], 64, 2, 1, 16, sinks=True)


@pytest.mark.parametrize("D", DIMS)
def test_large_scores(D):
    """Scores far apart: the running maximum moves, most probabilities vanish."""
    compare([700, 50], [1, 9], D, 4, 2, 16, scale=3.0, k_std=4.0, seed=4)
    compare([700, 50], [1, 9], D, 4, 2, 16, scale=-1.0, seed=5)
    compare([60], [3], D, 4, 2, 16, scale=0.0, seed=6)


@pytest.mark.parametrize("new", [1, 40])
def test_queries_of_any_size(new):
    """Rows of q far apart in size, zeros among them: each has its own power of two."""
    m = _m()
    b = Batch([100], 128, 2, 16)
    q = queries(new, 8, 128, 1) * (10.0 ** torch.arange(-12, 4, 2)).view(1, 8, 1)
    q = q.to(BF16)
    q[:, 3] = 0
    out, lse = run(m, b, q, [new], return_lse=True)
    want = b.want(q, [0, new], 1 / math.sqrt(128))
    check(out, want[0], want[2])
    check_lse(lse, want[1], want[3])


@pytest.mark.parametrize("new", [1, 3, 40])
def test_not_finite(new):
    """A NaN key makes the queries that see it NaN, and only those; NaN in a query stays in its row."""
    m = _m()
    lengths, D = [90, 90], 128
    b = Batch(lengths, D, 2, 16)
    q = queries(2 * new, 8, D, 1)
    q[0, 5, 3], q[new, 1, 7] = float("nan"), float("inf")
    poisoned = 90 - new // 2 - 1  # seen by the later queries of the second request
    page = int(b.tables[1, poisoned // 16])
    b.cache[page, 1, 0, 0, 8 * D + poisoned % 16 * (D // 16):][:D // 16] = 0x7f  # its key, head 1
    out = run(m, b, q, [new, new]).cpu()
    bad = torch.zeros(2 * new, 8, dtype=torch.bool)
    bad[0, 5] = bad[new, 1] = True
    for i in range(new):
        if 90 - new + i >= poisoned:
            bad[new + i, 4:] = True
    assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)


@pytest.mark.parametrize("new", [1, 40])
def test_values_nan_scales_and_bad_pages(new):
    m = _m()
    D = 64
    b = Batch([100, 50], D, 1, 16)
    q = queries(2 * new, 2, D, 1)
    page = int(b.tables[0, 2])
    b.cache[page, 0, 0, 1, :8 * D], b.cache[page, 0, 0, 1, 8 * D:] = 0x22, 0x7f  # the values of tokens 32 .. 47
    b.v[0][32:48] = 448
    for wrong in (-1, b.cache.shape[0], 2 ** 31 - 1):
        tables = b.tables.clone()
        tables[1, 1] = wrong
        out = m.fp4_attention(q.cuda(), b.cache.cuda(), tables.cuda(), ints(b.lengths), ints([0, new, 2 * new]))
        want = b.want(q, [0, new, 2 * new], 1 / 8)
        check(out[:new], want[0][:new], want[2][:new])
        sees = torch.tensor([50 - new + i >= 16 for i in range(new)])
        assert torch.equal(out[new:].isnan().all(-1).all(-1).cpu(), sees)
        assert torch.equal(out[new:].isnan().any(-1).any(-1).cpu(), sees)


def test_strides_and_out():
    """q as a slice of a projection, out by heads, other rows of out left alone; workspaces of one's own."""
    m = _m()
    D, Hq, new = 128, 6, [1, 30, 2]
    b = Batch([50, 60, 70], D, 2, 32)
    q = queries(33, Hq, D, 3)
    wide = torch.zeros(33, Hq, 2 * D, dtype=BF16, device="cuda")
    wide[..., :D] = q.cuda()
    store = torch.full((Hq, 40, D), 7.0, dtype=BF16, device="cuda")
    ws = m.alloc_fp4_attention_workspace(8, Hq, 2, D)
    out = store.transpose(0, 1)[:33]
    got = m.fp4_attention(wide[..., :D], b.cache.cuda(), torch.cat([b.tables, b.tables], 1).cuda()[:, :b.tables.shape[1]],
                          ints(b.lengths), ints(sums(new)), out=out, workspace=ws)
    assert got is out
    want = b.want(q, sums(new), 1 / math.sqrt(D))
    check(out, want[0], want[2])
    assert (store[:, 33:] == 7).all()


def test_same_results_again():
    m = _m()
    for lengths, new in (([5000, 3, 800], [1, 1, 1]), ([900, 300], [200, 77])):
        b = Batch(lengths, 128, 2, 64)
        q = queries(sum(new), 16, 128, 1)
        first = run(m, b, q, new)
        for _ in range(5):
            assert torch.equal(run(m, b, q, new), first)


def test_stream_argument_and_graph():
    m = _m()
    for new in ([1, 1], [100, 3]):
        b = Batch([500, 120], 128, 2, 16)
        q, args = queries(sum(new), 8, 128, 2).cuda(), None
        args = (b.cache.cuda(), b.tables.cuda(), ints(b.lengths), ints(sums(new)))
        want = m.fp4_attention(q, *args)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = m.fp4_attention(q, *args, stream=s)
        s.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = m.fp4_attention(q, *args)
        q.copy_(-q)
        out.zero_()
        graph.replay()
        assert torch.equal(out, m.fp4_attention(q, *args))


def test_refusals():
    m = _m()
    b = Batch([20, 30], 64, 2, 16)
    q = torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    good = dict(q=q, cache=b.cache.cuda(), tables=b.tables.cuda(), lengths=ints([20, 30]), offsets=ints([0, 1, 2]))
    m.fp4_attention(**good)
    for bad in (dict(q=q.half()), dict(tables=b.tables.long().cuda()), dict(lengths=torch.zeros(2, device="cuda")),
                dict(offsets=ints([0, 1, 2]).long()), dict(sinks=torch.zeros(4, dtype=BF16, device="cuda")),
                dict(cache=b.cache.cuda().int()), dict(out=q.float())):
        with pytest.raises(TypeError):
            m.fp4_attention(**(good | bad))
    for bad in (dict(q=q[0]), dict(q=q[..., :32]), dict(tables=b.tables[:1].cuda()), dict(tables=b.tables.t().contiguous().t().cuda()),
                dict(lengths=ints([20, 30, 1])), dict(offsets=ints([0, 1])), dict(sinks=torch.zeros(3, device="cuda")),
                dict(window=-1), dict(window=2 ** 31), dict(out=q[:1]), dict(cache=b.cache), dict(q=q.cpu()),
                dict(workspace=torch.zeros(1 << 24, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            m.fp4_attention(**(good | bad))
    for bad in (dict(scale=float("inf")), dict(k_scale=-1.0), dict(v_scale=0.0), dict(q=q[:, :3]),
                dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                dict(workspace=torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")[16:])):
        with pytest.raises(m.MoeFp4Error):
            m.fp4_attention(**(good | bad))
