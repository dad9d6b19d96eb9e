"""fa_fwd_paged: how exact the weights of a decoding tile are, requests that the
tensors cut, against float64; and batches that are mostly empty."""
from __future__ import annotations

import math

import pytest
import torch

import exact_attention_113_b200 as fa
from tests import paged_reference as ref
from tests.test_paged_gpu import Batch

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SEEN = 1 / math.sqrt(64)


def _exact_weights_bound(out, mag, total, dtype):
    """Where a weight is kept as the sum of two 16-bit values: half a step of
    the result, 2^-13 of mag for fp32 scores (see attention_bound), and half a
    step of half a step of each weight; fp16's smallest step is 2^-24."""
    h = ref.HALF[dtype]
    b = h * (1 + 2.0 ** -6) * out.abs() + (2.0 ** -13 + h * h) * mag
    if dtype == F16:
        b = b + 2.0 ** -25 * total + 2.0 ** -25
    return b


# up to 8 rows (new tokens x heads of a group) a request
@pytest.mark.parametrize("H,H_kv,D,q_lens", [
    (8, 1, 128, [1, 1, 1, 1]), (8, 2, 64, [1, 2, 1, 2]), (4, 4, 128, [1, 8, 5, 1]),
    (3, 3, 48, [1, 1, 3, 8]), (7, 1, 16, [1, 1, 1, 1]), (4, 2, 96, [4, 1, 3, 2]),
])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("wl", [-1, 40])
def test_weights_of_decoding_rows(H, H_kv, D, q_lens, dtype, wl):
    b = Batch(q_lens, [3 + n for n in q_lens[:1]] + [20, 131, 1200], H, H_kv, D, dtype, 16, seed=H * D)
    out, lse = b.run(window_left=wl)
    b.check(out, lse, wl=wl)
    clean = [torch.nan_to_num(c, nan=0.0) for c in (b.k, b.v)]
    want, _, mag, total = ref.attention(b.q, *clean, b.table, b.cu_q, b.kv_lens, 1 / math.sqrt(D),
                                        True, wl, -1)
    real = int(b.cu_q[-1])
    bound = _exact_weights_bound(want, mag, total, dtype)
    assert ((out.double() - want).abs() <= bound)[:real].all()


def test_weights_of_one_request_cut_over_all_ctas():
    # values that cancel: the result is small beside its terms
    b = Batch([1], [30000], 8, 1, 128, BF16, 16, seed=5)
    out, lse = b.run()
    clean = [torch.nan_to_num(c, nan=0.0) for c in (b.k, b.v)]
    want, _, mag, total = ref.attention(b.q, *clean, b.table, b.cu_q, b.kv_lens, 1 / math.sqrt(128),
                                        True, -1, -1)
    assert ((out.double() - want).abs() <= _exact_weights_bound(want, mag, total, BF16))[:1].all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_infinite_values_of_visible_keys(D, dtype):
    # equal scores: every weight is 1, and exact, so its rest is 0
    b = Batch([1, 2, 1], [7, 300, 40], 8, 2, D, dtype, 16, seed=33)
    b.q.zero_()
    want, _ = b.run()
    spots = ((0, 3, 1, math.inf), (1, 150, 0, -math.inf), (2, 39, 0, math.inf))
    for r, key, head, x in spots:
        page, row = int(b.table[r, key // 16]), key % 16
        b.v[page, row, head, 5] = x
    out, lse = b.run()
    assert torch.isfinite(lse[: int(b.cu_q[-1])]).all()
    for r, key, head, x in spots:
        rows, heads = slice(int(b.cu_q[r]), int(b.cu_q[r + 1])), slice(4 * head, 4 * head + 4)
        assert (out[rows, heads, 5] == x).all()
        want[rows, heads, 5] = x
    assert torch.equal(out, want)


# ------------------------------------------------------------ cut requests
def _close(out, lse, want, dtype):
    o, e, mag, total = want
    assert ((out.double() - o).abs() <= ref.attention_bound(o, mag, total, dtype)).all()
    seen = torch.isfinite(e)
    assert torch.equal(torch.isneginf(lse), ~seen)
    assert ((lse.double() - e)[seen].abs() <= ref.LSE_BOUND).all()


@pytest.mark.parametrize("wl", [-1, 70])
@pytest.mark.parametrize("rows", [50, 73, 3, 330])
def test_rows_of_a_request_that_total_q_cuts(rows, wl):
    # the last request's new tokens do not all have a row: those that have one
    # keep their places, and see no key behind them
    b = Batch([2, 40, 300], [90, 40, 700], 4, 2, 64, F16, 16, seed=60, pad_rows=0)
    clean = [torch.nan_to_num(c, nan=0.0) for c in (b.k, b.v)]
    want = ref.attention(b.q, *clean, b.table, b.cu_q, b.kv_lens, SEEN, True, wl, -1)
    out, lse = fa.flash_fwd_paged(b.q[:rows], b.k, b.v, b.table, b.cu_q, b.kv_lens, window_left=wl)
    _close(out, lse, [t[:rows] for t in want], F16)


def test_keys_behind_a_table_that_is_too_narrow():
    # positions 100 .. 199 over a table of 128 tokens: the keys that it holds,
    # each token at its own place
    b = Batch([100], [200], 4, 2, 64, BF16, 16, seed=61, pad_rows=0)
    clean = [torch.nan_to_num(c, nan=0.0) for c in (b.k, b.v)]
    out, lse = fa.flash_fwd_paged(b.q, b.k, b.v, b.table[:, :8].clone(), b.cu_q, b.kv_lens)

    def part(rows, kv, causal):
        q = b.q[rows]
        cu = torch.tensor([0, q.shape[0]], dtype=torch.int32, device="cuda")
        n = torch.tensor([kv], dtype=torch.int32, device="cuda")
        return ref.attention(q, *clean, b.table, cu, n, SEEN, causal, -1, -1)
    _close(out[:28], lse[:28], part(slice(0, 28), 128, True), BF16)
    _close(out[28:], lse[28:], part(slice(28, 100), 128, False), BF16)


def test_step_over_its_capacity():
    # page tables for more tokens than the batch has rows, then the attention
    lens, ctx, page, T, H, H_kv, D = [30, 50, 60], [10, 100, 7], 16, 100, 4, 2, 64
    full = Batch(lens, [a + c for a, c in zip(lens, ctx)], H, H_kv, D, BF16, page, seed=62, pad_rows=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    p = fa.paged_plan(torch.tensor(lens, **i32), torch.tensor(ctx, **i32), full.table.clone(),
                      torch.arange(40, **i32), page, T)
    assert p.cu_q.tolist() == [0, 30, 80, 140] and p.positions.tolist()[80:] == list(range(7, 27))
    out, lse = fa.flash_fwd_paged(full.q[:T], full.k, full.v, full.table, p.cu_q, p.kv_lens)
    clean = [torch.nan_to_num(c, nan=0.0) for c in (full.k, full.v)]
    want = ref.attention(full.q, *clean, full.table, full.cu_q, full.kv_lens, SEEN, True, -1, -1)
    _close(out, lse, [t[:T] for t in want], BF16)


# ------------------------------------------------------------ empty requests
@pytest.mark.parametrize("n,B,kind", [
    (8, 512, "behind"), (8, 512, "before"), (8, 600, "spread"), (300, 5000, "spread"),
    (1, 4000, "between"), (300, 1 << 20, "spread"), (2, 1 << 20, "behind"),
])
def test_mostly_empty_batches(n, B, kind):
    # the same bits as the requests alone: the work is cut in the same places
    g = torch.Generator().manual_seed(n)
    q = torch.randint(1, 20, (n,), generator=g).tolist()
    kv = [x + int(y) for x, y in zip(q, torch.randint(0, 300, (n,), generator=g))]
    b = Batch(q, kv, 4, 2, 64, F16, 16, seed=70)
    want = b.run()
    at = {"behind": torch.arange(n), "before": torch.arange(B - n, B),
          "between": torch.full((n,), B // 2),
          "spread": torch.linspace(0, B - 1, n).long()}[kind]
    lens = torch.zeros(B, dtype=torch.int32)
    lens[at] = torch.tensor(q, dtype=torch.int32)
    kvs = torch.full((B,), 33, dtype=torch.int32)       # empty requests may have a cache
    kvs[at] = b.kv_lens.cpu()
    table = torch.full((B, b.table.shape[1]), -1, dtype=torch.int32, device="cuda")
    table[at.cuda()] = b.table
    b.cu_q = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0).int()]).cuda()
    b.kv_lens, b.table = kvs.cuda(), table
    got = b.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_strides_of_one_element_axes():
    # one token, one head, one K/V head, one page
    for H, H_kv, T, kv in ((8, 2, 1, 300), (1, 1, 5, 200), (4, 1, 1, 9)):
        b = Batch([T], [kv], H, H_kv, 64, BF16, 256 if H == 4 else 16, seed=80, pad_rows=0)
        want, want_lse = b.run()

        def odd(x):
            return x.as_strided(x.shape, [n if x.shape[a] > 1 else 3 for a, n in enumerate(x.stride())])
        out = odd(torch.full_like(b.q, 3.0))
        _, lse = fa.flash_fwd_paged(odd(b.q), odd(b.k), odd(b.v), b.table, b.cu_q, b.kv_lens, out=out)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
