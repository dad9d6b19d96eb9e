"""fa_paged_plan after the free list has run out: exact integers."""
from __future__ import annotations

import pytest
import torch

import exact_attention_113_b200 as fa
from tests.test_plan_gpu import _t

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
