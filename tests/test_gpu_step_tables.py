"""GPU: block tables and slot maps from request lengths, against one request
after another (step_reference.py)."""
import random

import pytest
import torch

import linear_exl3_input_amd as ex
import step_reference as step
from gpu_util import banner

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(pages, page):
    return ex.KvCache.empty(pages, page, 1, 64, 4)


def check(c, q, kv, table, free, tokens, taken=None, out=None):
    want = step.extended(c.pages, c.page_size, q, kv, table, free, tokens, taken or 0)
    t = ints(table) if table else torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    args = (ints(q), ints(kv), t, ints(free))
    got = ex.cache_extend(c, *args, tokens, None if taken is None else ints([taken]), out)
    for name, g, w in zip((*ex.CacheStep._fields, "table"), (*got, t), want):
        assert g.tolist() == w, name
    assert args[0].tolist() == q and args[1].tolist() == kv and args[3].tolist() == free
    return got, t


def batch(r, n, page, q_max, kv_max, width=None, hole=0.0):
    """Lengths, a table whose rows hold what they need, and the free pages."""
    kv = [r.choice((0, r.randrange(kv_max + 1), r.randrange(1 + kv_max // page) * page)) for _ in range(n)]
    q = [r.choice((0, 1, r.randrange(q_max + 1))) for _ in range(n)]
    width = width or -(-(kv_max + q_max) // page)
    pages = sum(-(-(a + b) // page) for a, b in zip(q, kv)) + 3
    order = list(range(pages))
    r.shuffle(order)
    at, table = 0, []
    for b in kv:
        have = min(width, -(-b // page))
        table.append([-1 if r.random() < hole else order[at + i] for i in range(have)] + [-7] * (width - have))
        at += have
    return cache(pages, page), q, kv, table, order[at:]


@pytest.mark.parametrize("n,page,q_max,kv_max", [(1, 16, 1, 0), (1, 64, 1, 63), (64, 64, 1, 9000), (7, 16, 300, 1000), (255, 32, 3, 500),
                                                (256, 16, 40, 100), (257, 128, 2, 3000), (1000, 1024, 90, 5000)])
def test_tables(n, page, q_max, kv_max):
    banner(f"tables of {n} requests, pages of {page}")
    r = random.Random(n)
    c, q, kv, table, free = batch(r, n, page, q_max, kv_max)
    total = sum(q)
    for tokens in sorted({total, total + 13, total // 2, 0}):
        check(c, q, kv, table, free, tokens)


def test_more_rows_than_a_launch_has_threads():
    c, q, kv, table, free = batch(random.Random(1), 700, 16, 1500, 700)
    assert sum(q) > 512 * 256
    check(c, q, kv, table, free, sum(q) + 5)


def test_too_few_free_pages_and_pages_taken_before():
    r = random.Random(2)
    c, q, kv, table, free = batch(r, 40, 16, 60, 200)
    full, _ = check(c, q, kv, table, free, sum(q))
    need = int(full.counts[1])
    for n in (0, 1, need - 1, need):
        got, t = check(c, q, kv, table, free[:n], sum(q))
        assert int(got.counts[1]) == need
    for taken in (-3, 0, 5, len(free) - 1, len(free), 2 ** 31 - 1):
        check(c, q, kv, table, free, sum(q), taken)


def test_holes_narrow_tables_and_pages_that_are_none():
    r = random.Random(3)
    c, q, kv, table, free = batch(r, 30, 16, 50, 400, hole=0.3)
    check(c, q, kv, table, free, sum(q))
    c, q, kv, table, free = batch(r, 30, 16, 50, 400, width=9)
    check(c, q, kv, table, free, sum(q))
    c, q, kv, table, free = batch(r, 30, 16, 50, 400)
    check(c, q, kv, [[x + 2 if x >= 0 else x for x in row] for row in table], [x if x % 3 else x + 2 ** 30 for x in free], sum(q))


def test_lengths_out_of_range():
    c = cache(10, 16)
    big = 2 ** 31 - 1
    check(c, [-5, 3, big, 1], [4, -9, 5, big], [[1, 2, 3]] * 4, [7, 8, 9], 30)
    check(c, [big] * 300, [0] * 300, [[0]] * 300, [1], 20)
    check(c, [2 ** 20] * 4000, [0] * 4000, [[0]] * 4000, [1], 20)  # more rows wanted than 32 bits count


def test_no_requests_no_rows_no_table():
    c = cache(10, 16)
    check(c, [], [], [], [1, 2], 5)
    check(c, [], [], [], [], 0)
    t = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    got = ex.cache_extend(c, ints([3, 2]), ints([0, 5]), t, ints([]), 5)
    assert got.slots.tolist() == [-1] * 5 and got.positions.tolist() == [0, 1, 2, 5, 6] and got.counts.tolist() == [5, 0]


def test_strided_tables_given_outputs_and_the_same_call_again():
    r = random.Random(4)
    c, q, kv, table, free = batch(r, 20, 16, 30, 100)
    n = sum(q)
    out = ex.CacheStep(*(torch.full((m,), -9, dtype=torch.int32, device="cuda") for m in (21, 20, n, n, 2)))
    got, t = check(c, q, kv, table, free, n, out=out)
    assert got is out
    wide = torch.full((20, len(table[0]) + 11), -5, dtype=torch.int32, device="cuda")
    view = wide[:, 4:4 + len(table[0])]
    view.copy_(ints(table))
    for _ in range(2):  # the second call finds the entries that the first one wrote
        again = ex.cache_extend(c, ints(q), ints(kv), view, ints(free), n)
        assert all(torch.equal(a, b) for a, b in zip(again, got)) and torch.equal(view, t)
    assert (wide[:, :4] == -5).all() and (wide[:, 4 + len(table[0]):] == -5).all()


def test_a_captured_loop_of_steps():
    """Requests grow token by token from one graph; each replay against the lengths counted here."""
    page, B = 16, 5
    c = cache(64, page)
    lens = [0, 15, 16, 31, 7]
    order = list(range(63, -1, -1))
    table = [[order[8 * b + i] if i < -(-n // page) else -1 for i in range(6)] for b, n in enumerate(lens)]
    used = {x for row in table for x in row}
    free = [x for x in order if x not in used]
    t, fr, kv, one = ints(table), ints(free), ints(lens), ints([1, 1, 0, 1, 1])
    taken = ints([0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s = ex.cache_extend(c, one, kv, t, fr, 6, taken)
        kv.copy_(s.kv_len)
        taken.add_(s.counts[1:])
    want_taken = 0
    for i in range(40):
        graph.replay()
        torch.cuda.synchronize()
        want = step.extended(64, page, [1, 1, 0, 1, 1], lens, table, free, 6, want_taken)
        lens, table = want[1], want[5]
        want_taken += want[4][1]
        assert [x.tolist() for x in s] == list(want[:5]) and t.tolist() == table, f"replay {i}"
        assert kv.tolist() == lens and taken.tolist() == [want_taken]
