"""Plans whose work is in pages, not in tokens: long requests that end, with few new tokens or none, in place and out of it."""
from __future__ import annotations

import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import step_reference as ref  # noqa: E402
from test_gpu_step import Plan, lib  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_sparse_attention_08_gb300 import _build
    _build.build()


def ending(r, B, ends, pages, page, *, new=True, total=None, free=0, **kw):
    """B requests of up to `pages` pages, of which `ends` are over and give back all but what they share."""
    over = set(r.sample(range(B), ends))
    held = [pages if s in over else r.randint(1, pages) for s in range(B)]
    kv = [0 if s in over else r.randint(max(0, (h - 1) * page), h * page) for s, h in enumerate(held)]
    ns = [0 if s in over else r.randint(0, 2) for s in range(B)] if new else None
    shared = [r.choice([0, 0, 1]) for _ in range(B)]
    ids = list(range(sum(held) + free))
    r.shuffle(ids)
    table = [[ids.pop() if j < h else -9 for j in range(pages + 2)] for h in held]
    cap = sum(held) + free + 5
    return Plan(ns, kv, held, shared, None, table, ids + [-5] * (cap - len(ids)), len(ids), page=page, pool=cap,
                total=(sum(ns or [0]) if total is None else total), **kw)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B, ends, pages", [(4, 1, 8192), (128, 128, 1024), (100, 3, 700), (2048, 2000, 40), (129, 1, 3000)])
def test_long_requests_end_beside_few_tokens(B, ends, pages, in_place):
    """The lists are as long as the tables, so the whole device goes through them, not one CTA."""
    p = ending(random.Random(B), B, ends, pages, 16, in_place=in_place)
    p.call()
    assert lib().dsv4_last_launch_count() == 2
    _, err = p.check()
    assert err == 0


@pytest.mark.parametrize("B, pages", [(16, 5000), (600, 70)])
@pytest.mark.parametrize("total", [0, 9])
def test_pages_are_only_given_back(B, pages, total):
    p = ending(random.Random(B), B, B // 2, pages, 16, new=False, total=total, optional=False)
    p.call()
    assert lib().dsv4_last_launch_count() == 2
    want, err = p.check()
    assert err == 0 and want["count"] > pages


def test_what_is_given_back_is_taken_at_once_by_many():
    """The whole device: nothing free, one long request ends, the pages of 300 others' new rows come from it."""
    r = random.Random(3)
    B, page, width = 301, 8, 700
    held = [width] + [2] * (B - 1)
    kv, new = [0] + [r.randint(9, 16) for _ in range(B - 1)], [0] + [r.randint(0, 16) for _ in range(B - 1)]
    ids = list(range(sum(held)))
    r.shuffle(ids)
    table = [[ids.pop() if j < h else -9 for j in range(width)] for h in held]
    p = Plan(new, kv, held, None, [7] * B, table, [-5] * sum(held), 0, page=page, pool=sum(held), total=sum(new), in_place=True)
    p.call()
    want, err = p.check()
    assert err == 0 and want["count"] == width - sum(max(0, -(-(a + b) // page) - 2) for a, b in zip(kv[1:], new[1:]))


def test_a_small_step_is_one_launch():
    p = ending(random.Random(2), 16, 2, 20, 64, total=64, free=30)
    p.call()
    assert lib().dsv4_last_launch_count() == 1
    assert p.check()[1] == 0


@pytest.mark.parametrize("B", [5, 200])
@pytest.mark.parametrize("total", [255, 256, 257, 2049])
@pytest.mark.parametrize("cap", [4095, 4096, 4097])
def test_both_forms_at_their_border(B, total, cap):
    """Either side of the sizes up to which one launch does all: the same results."""
    r = random.Random(cap + B)
    page, width = 8, 4200 // B + 30
    held = [4000 // B] * B
    kv, new = [0 if s % 2 else h * page - 3 for s, h in enumerate(held)], [s % 3 for s in range(B)]
    ids = list(range(sum(held) + 90))
    r.shuffle(ids)
    table = [[ids.pop() if j < h else -9 for j in range(width)] for h in held]
    p = Plan(new, kv, held, None, None, table, ids + [-5] * (cap - len(ids)), len(ids), page=page, pool=sum(held) + 90, total=total)
    p.call()
    want, err = p.check()
    assert err == 0 and want["count"] > 90


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("what", ["returned", "returned_high", "taken", "passed_on"])
def test_a_page_outside_the_pool_is_flagged_when_it_moves(what, wide):
    """When it goes to the stack or comes from it, also where no row of the step lies on it; everything else is as if it were
    a page."""
    page, width = 16, 5000 if wide else 6
    new, kv, held = [0, 0, 1], [0, 20, 16], [3, 2, 1]
    table = [[1, 2, 3], [4, 5], [6]]
    free, count = [7, 8, 9], 3
    if what == "returned":
        table[0][1] = -1
    if what == "returned_high":
        table[0][2] = 4200
    if what == "taken":                                               # for rows that were there before: no new token on it
        new, kv, held, free[2] = [0, 0, 0], [40, 20, 17], [3, 2, 1], -3
    if what == "passed_on":                                           # from an ended request straight to another's old rows
        new, kv, held, count = [0, 0, 0], [0, 20, 17], [1, 2, 1], 0
        table[0][0] = 4200
    table = [row + [-9] * (width - len(row)) for row in table]
    free = free[:count] + [-5] * ((4200 if wide else 12) - count)
    p = Plan(new, kv, held, None, None, table, free, count, page=page, pool=4200, total=4)
    p.call()
    assert lib().dsv4_last_launch_count() == (2 if wide else 1)
    want, err = ref.plan(*p.lists, **p.kw)
    # (the plain form looks at the rows' pages alone: the page of the one new row is the last that was given back)
    assert err == (ref.BAD_INDEX if what == "returned_high" else 0)
    assert lib().dsv4_read_error_word(p.ws)[1] == ref.BAD_INDEX
    for k, t in dict(cu_q=p.cu, slots=p.slots, table=p.table, free=p.free, kv_len=p.kv_out, held=p.held_out).items():
        assert t.tolist() == want[k], k
    assert p.count_out.tolist() == [want["count"]]


def test_pages_that_do_not_fit_the_stack_stay_in_the_table():
    p = Plan([0, 0], [5, 0], [4, 3], None, None, [[1, 2, 3, 4], [5, 6, 7, -9]], [8, 9, -5, -5], 2, page=16, pool=10, total=0)
    p.call()
    want, err = p.check()
    assert err == ref.BAD_INDEX and want["free"] == [8, 9, 2, 3] and want["held"] == [1, 0]
    assert p.table.tolist() == [[1, 2, 3, 4], [5, 6, 7, -9]]
