"""fa_paged_plan where its scan takes several tiles of requests, and after the
free list has run out: exact integers."""
from __future__ import annotations

import pytest
import torch

import exact_attention_113_b200 as fa
from tests import paged_reference as ref
from tests.test_plan_gpu import _case, _check, _t

pytestmark = pytest.mark.gpu


def _step(q, c, table, free, page, T):
    """One call on the GPU; the table as it is afterwards."""
    dt = _t(table)
    p = fa.paged_plan(_t(q), _t(c), dt, _t(free), page, T)
    return p, dt.tolist()


def test_tokens_behind_a_shortage_are_counted():
    # step 1 leaves table entries of -1; the tokens that step 2 puts behind them
    # in the same pages have no slot either
    page, free = 16, [5]
    p, table = _step([20, 20], [0, 0], [[-1] * 4, [-1] * 4], free, page, 40)
    assert p.counts.tolist() == [40, 1, 24]
    assert (p.slots < 0).sum() == 24
    p, table = _step([3, 14], p.kv_lens.tolist(), table, [7, 8], page, 20)
    assert p.positions.tolist() == [20, 21, 22, *range(20, 34), -1, -1, -1]
    # request 0: three in page 1 (-1); request 1: twelve there, two in its new page
    assert p.slots.tolist() == [-1] * 15 + [7 * 16, 7 * 16 + 1] + [-1] * 3
    assert p.counts.tolist() == [17, 1, 15]
    assert table[0][:3] == [5, -1, -1] and table[1][:3] == [-1, -1, 7]


@pytest.mark.parametrize("q,ctx,row,want", [
    (1, 17, [3, -1, -1], 1),      # a single token into a page that is not there
    (15, 17, [3, -1, -1], 15),    # all that is left of it
    (16, 17, [3, -1, -1], 15),    # and one in the next page
    (0, 17, [3, -1, -1], 0),      # no new token
    (4, 16, [-1, -1, -1], 0),     # full pages that are not there do not count
    (4, 15, [-1, -1, -1], 1),
    (9, 47, [1, 2, -1], 9),       # the last column, and tokens beyond the table
    (9, 50, [1, 2, -1], 9),       # the cache itself passes the table
])
def test_count_of_tokens_without_a_slot(q, ctx, row, want):
    p, _ = _step([2, q, 1], [0, ctx, 3], [[-1] * 3, row, [0, -1, -1]], [10, 11, 12], 16, q + 3)
    assert int((p.slots < 0).sum()) == want
    assert p.counts.tolist()[2] == want


# 1024 requests a tile: its borders, several tiles, and one block (few tokens)
# or many of them
@pytest.mark.parametrize("B", [1023, 1024, 1025, 2047, 2049, 3000])
@pytest.mark.parametrize("chunk,ctx,page", [(1, 90, 16), (11, 200, 32)])
def test_tiles_of_requests(B, chunk, ctx, page):
    case = _case(B + chunk, B, chunk, ctx, page)
    _check(*case, sum(case[0]) + 5)


def test_tile_border_without_new_tokens():
    q, c, table, free, page = _case(31, 2500, 7, 100, 16)
    for i in (*range(1000, 1040), *range(2040, 2060), 2499):
        q[i] = 0
    _check(q, c, table, free, page, sum(q) + 1100)


def test_one_block_walks_all_tiles():
    # fewer tokens than a block serves
    q = [0] * 5000
    c = [i % 40 for i in range(5000)]
    for i in (0, 1023, 1024, 2048, 4999):
        q[i] = 33
    table = [[3 * i, 3 * i + 1, 3 * i + 2, -1, -1] for i in range(5000)]
    _check(q, c, table, list(range(20000, 20040)), 16, sum(q) + 2)


@pytest.mark.parametrize("share", [0.3, 0.7])
def test_free_list_runs_out_in_a_later_tile(share):
    q, c, table, free, page = _case(41, 2049, 40, 60, 16)
    free = free[: int(share * len(free))]
    _check(q, c, table, free, page, sum(q))


def test_capacity_ends_in_the_second_tile():
    q, c, table, free, page = _case(51, 2049, 20, 60, 16)
    _check(q, c, table, free, page, sum(q[:1500]))
    want = ref.plan(q, c, table, free, page, sum(q))
    assert want[5][2] == 0
