"""cache_step against the same step written request by request."""
import random

import pytest
import torch

from tests.gpu_util import ensure_built

pytestmark = pytest.mark.gpu


def _m():
    ensure_built()
    import fp4_weight_moe_gb300 as m
    return m


def plain(lengths, new, tables, free, count, page, tokens, finished):
    tables, free = [list(t) for t in tables], list(free)
    W, R = len(tables[0]) if tables else 0, len(lengths)
    up = lambda n: -(-n // page)  # noqa: E731
    lengths, new = [max(n, 0) for n in lengths], [max(n, 0) for n in new]
    top = min(max(count, 0), len(free))
    for r in range(R):
        if finished[r]:
            for j in range(min(up(lengths[r]), W)):
                if top < len(free):
                    free[top] = tables[r][j]
                    top += 1
            lengths[r] = 0
    asked, taken = 0, 0
    accepted, out, where, pos = [], [], [], []
    for r in range(R):
        have, all_ = up(lengths[r]), up(lengths[r] + new[r])
        wide = all_ > W and new[r] > 0
        need = 0 if wide else all_ - have
        fits = not wide and (need == 0 or asked + need <= top)
        if fits:
            for j in range(need):
                tables[r][have + j] = free[top - 1 - asked - j]
            taken += need
        asked += need
        accepted.append(new[r] if fits else 0)
        out.append(lengths[r] + accepted[-1])
        for i in range(new[r]):
            p = lengths[r] + i
            pos.append(p)
            where.append(tables[r][p // page] * page + p % page if fits else -1)
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    pos, where = pos[:tokens], where[:tokens]
    pos += [0] * (tokens - len(pos))
    where += [-1] * (tokens - len(where))
    return offsets, pos, where, out, [top - taken], accepted, tables, free


def state(R, page, ctx, new, seed, spare, extra_width=1, ends=0.2):
    rng = random.Random(seed)
    lengths = [rng.choice([0, 1, page - 1, page, rng.randint(0, ctx)]) for _ in range(R)]
    fresh = [rng.choice([0, 1, new, rng.randint(0, new)]) for _ in range(R)]
    have = [-(-n // page) for n in lengths]
    width = max([-(-(n + f) // page) for n, f in zip(lengths, fresh)] + [0]) + extra_width
    pool = list(range(sum(have) + spare))
    rng.shuffle(pool)
    tables, at = [], 0
    for h in have:
        tables.append((pool[at:at + h] + [-1] * width)[:max(width, 0)])
        at += h
    free = pool[at:] + [-7] * sum(have)
    finished = [rng.random() < ends for _ in range(R)]
    return lengths, fresh, tables, free, spare, finished


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def run_and_compare(m, s, page, tokens, in_place=False, bool_mask=True):
    lengths, fresh, tables, free, count, finished = s
    want = plain(lengths, fresh, tables, free, count, page, tokens, finished)
    R = len(lengths)
    t_len, t_count = ints(lengths), ints([count])
    t_tab = ints(tables) if R else torch.empty(0, 4, dtype=torch.int32, device="cuda")
    t_free = ints(free)
    mask = ints(finished, torch.bool if bool_mask else torch.uint8)
    more = dict(lengths_out=t_len, free_count_out=t_count) if in_place else {}
    got = m.cache_step(t_len, ints(fresh), t_tab, t_free, t_count, page, tokens,
                       finished=mask if any(finished) else None, **more)
    assert got.offsets.tolist() == want[0]
    assert got.positions.tolist() == want[1]
    assert got.slots.tolist() == want[2]
    assert got.lengths.tolist() == want[3]
    assert got.free_count.tolist() == want[4]
    assert got.accepted.tolist() == want[5]
    if R:
        assert t_tab.tolist() == want[6]
    assert t_free.tolist() == want[7]
    if in_place:
        assert got.lengths is t_len and got.free_count is t_count
    else:
        assert t_len.tolist() == lengths and t_count.tolist() == [count]
    return want


@pytest.mark.parametrize("R", [0, 1, 2, 31, 64, 513, 1024, 1025, 2500])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(R, page, in_place):
    m = _m()
    s = state(R, page, 300, 20, R + page, spare=2 * R + 5)
    run_and_compare(m, s, page, sum(s[1]), in_place, bool_mask=R % 2 == 0)


@pytest.mark.parametrize("new", [1, 700])
def test_many_tokens(new):
    """Past the tokens that one launch places, with rows behind the last."""
    m = _m()
    s = state(40, 32, 500, new, new, spare=2000)
    run_and_compare(m, s, 32, 40 * 700, in_place=True)


@pytest.mark.parametrize("spare", [0, 1, 3, 10])
def test_short_of_pages(spare):
    """Requests that the stack cannot serve are refused, those that need no page are not."""
    m = _m()
    for seed in range(6):
        s = state(20, 16, 200, 40, seed, spare, ends=0.1 if seed % 2 else 0.0)
        want = run_and_compare(m, s, 16, sum(s[1]) + 3)
    assert 0 in want[5]


def test_narrow_tables_and_few_tokens():
    m = _m()
    s = state(12, 16, 100, 60, 5, spare=100, extra_width=-2)
    want = run_and_compare(m, s, 16, sum(s[1]) // 2)
    assert any(f > 0 and a == 0 for f, a in zip(s[1], want[5]))


def test_negative_counts_and_a_deep_stack():
    m = _m()
    lengths, fresh, tables, free, count, finished = state(8, 16, 100, 10, 1, spare=30)
    fresh[3], lengths[4], tables[4] = -5, -1, [-1] * len(tables[4])
    s = (lengths, fresh, tables, free, len(free) + 10, [False] * 8)
    run_and_compare(m, s, 16, sum(max(f, 0) for f in fresh))


def test_strided_tables():
    m = _m()
    lengths, fresh, tables, free, count, _ = state(9, 16, 100, 10, 3, spare=30)
    want = plain(lengths, fresh, tables, free, count, 16, sum(fresh), [False] * 9)
    wide = torch.full((9, len(tables[0]) + 5), -9, dtype=torch.int32, device="cuda")
    view = wide[:, :len(tables[0])]
    view.copy_(ints(tables))
    got = m.cache_step(ints(lengths), ints(fresh), view, ints(free), ints([count]), 16, sum(fresh))
    assert got.slots.tolist() == want[2] and view.tolist() == want[6]
    assert (wide[:, len(tables[0]):] == -9).all()


def test_refusals():
    m = _m()
    i = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    good = dict(lengths=i(4), new_tokens=i(4), tables=i(4, 3), free_pages=i(9), free_count=i(1), page_size=16, tokens=4)
    m.cache_step(**good)
    for bad in (dict(lengths=i(4, d=torch.int64)), dict(new_tokens=i(4, d=torch.float32)), dict(tables=i(4, 3, d=torch.int64)),
                dict(finished=i(4))):
        with pytest.raises(TypeError):
            m.cache_step(**(good | bad))
    for bad in (dict(new_tokens=i(5)), dict(tables=i(3, 3)), dict(tables=i(3, 4).t()), dict(free_count=i(2)),
                dict(free_pages=i(3, 3)), dict(tokens=-1), dict(finished=i(3, d=torch.bool)), dict(lengths=i(2, 2)),
                dict(lengths_out=i(3)), dict(lengths=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            m.cache_step(**(good | bad))
    with pytest.raises(m.MoeFp4Error):
        m.cache_step(**(good | dict(page_size=20)))
