"""fa_paged_plan against a token-by-token plain form: exact integers."""
from __future__ import annotations

import random

import pytest
import torch

import exact_attention_113_b200 as fa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


def _t(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _case(seed, B, chunk, ctx, page, extra=2, free_less=0):
    r = random.Random(seed)
    q = [r.choice([0, 1, r.randint(0, chunk)]) for _ in range(B)]
    c = [r.randint(0, ctx) for _ in range(B)]
    width = max(-(-(a + b) // page) for a, b in zip(q, c)) + extra
    need = sum(-(-(a + b) // page) for a, b in zip(q, c))
    pages = list(range(need + 5))
    r.shuffle(pages)
    table = [[-1] * max(width, 1) for _ in range(B)]
    for b in range(B):
        for i in range(min(-(-c[b] // page), width)):
            table[b][i] = pages.pop()
    return q, c, table, pages[: max(0, len(pages) - 5 - free_less)], page


def _check(q, c, table, free, page, T):
    want = ref.plan(q, c, table, free, page, T)
    dt = _t(table)
    p = fa.paged_plan(_t(q), _t(c), dt, _t(free), page, T)
    got = (p.cu_q, p.kv_lens, p.positions, p.slots, dt, p.counts)
    for name, g, w in zip(("cu_q", "kv_lens", "positions", "slots", "table", "counts"), got, want):
        assert g.tolist() == w, name


@pytest.mark.parametrize("seed,B,chunk,ctx,page,pad", [
    (1, 1, 1, 0, 16, 0), (2, 1, 3000, 50, 16, 7), (3, 8, 1, 900, 16, 0), (4, 255, 5, 100, 32, 3),
    (5, 256, 40, 700, 16, 1), (6, 257, 40, 0, 64, 0), (7, 700, 9, 333, 128, 1500),
    (8, 3, 1, 40, 1, 0), (9, 5, 100, 100, 7, 2),
])
def test_plan(seed, B, chunk, ctx, page, pad):
    case = _case(seed, B, chunk, ctx, page)
    _check(*case, sum(case[0]) + pad)


def test_no_new_tokens():
    _check([0, 0, 0], [5, 0, 64], [[3, -1], [-1, -1], [4, -1]], [9], 64, 4)


def test_free_list_runs_out_and_is_empty():
    case = _case(11, 40, 200, 300, 16, free_less=25)
    _check(*case, sum(case[0]))
    _check([3, 20], [16, 0], [[1, -1], [-1, -1]], [], 16, 23)


def test_table_too_narrow():
    # request 0's new tokens pass the last column; request 1's cache already does
    _check([40, 3, 2], [10, 50, 0], [[0, -1, -1], [1, 2, 3], [-1, -1, -1]], [7, 8, 9], 16, 45)


def test_capacity_below_the_tokens():
    # positions and slots of the first num_tokens; everything else complete
    case = _case(12, 30, 100, 64, 16)
    _check(*case, sum(case[0]) // 2)


def test_negative_lengths_count_as_zero():
    _check([-3, 4], [2, -5], [[5, -1], [-1, -1]], [6, 7], 16, 5)


def test_strided_table_and_given_outputs():
    q, c, table, free, page = _case(13, 20, 60, 90, 16)
    T = sum(q) + 3
    want = ref.plan(q, c, table, free, page, T)
    width = len(table[0])
    wide = torch.full((20, width + 9), -7, dtype=torch.int32, device="cuda")
    wide[:, :width] = _t(table)
    out = fa.paged_plan(_t(q), _t(c), wide[:, :width].clone(), _t(free), page, T)
    for t in out:
        t.fill_(-9)
    p = fa.paged_plan(_t(q), _t(c), wide[:, :width], _t(free), page, T, out=out)
    assert p.slots.data_ptr() == out.slots.data_ptr()
    assert p.slots.tolist() == want[3] and wide[:, :width].tolist() == want[4]
    assert (wide[:, width:] == -7).all()


def test_graph_replay_with_other_lengths():
    q, c = _t([1, 1, 5]), _t([16, 3, 0])
    table, free = _t([[0, -1, -1], [1, -1, -1], [-1, -1, -1]]), _t([4, 5, 6, 7])
    out = fa.paged_plan(q, c, table, free, 16, 40)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.paged_plan(q, c, table, free, 16, 40, out=out)
    q.copy_(_t([2, 20, 0]))
    c.copy_(_t([15, 3, 0]))
    table.copy_(_t([[0, -1, -1], [1, -1, -1], [-1, -1, -1]]))
    want = ref.plan([2, 20, 0], [15, 3, 0], table.tolist(), free.tolist(), 16, 40)
    g.replay()
    torch.cuda.synchronize()
    got = (out.cu_q, out.kv_lens, out.positions, out.slots, table, out.counts)
    assert [t.tolist() for t in got] == list(want)


def test_alternating_outputs_and_refused_overlap():
    # each step's contexts are the lengths that the step before it wrote
    q, table = _t([1, 30, 2]), torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    free, c = _t(list(range(24))), _t([0, 0, 0])
    outs = [fa.paged_plan(_t([0] * 3), c, table, free, 16, 33) for _ in range(2)]
    rows, ctx, taken = table.tolist(), [0, 0, 0], 0
    for step in range(4):
        p = fa.paged_plan(q, c, table, free[taken:].clone(), 16, 33, out=outs[step % 2])
        want = ref.plan([1, 30, 2], ctx, rows, list(range(24))[taken:], 16, 33)
        assert p.slots.tolist() == want[3] and table.tolist() == want[4]
        assert p.kv_lens.tolist() == want[1] and p.counts.tolist() == want[5]
        c, ctx, rows = p.kv_lens, want[1], want[4]
        taken += want[5][1]
    with pytest.raises(fa.FaError):
        fa.paged_plan(q, outs[0].kv_lens, table, free, 16, 33, out=outs[0])
