"""fa_fwd_paged: how exact the weights of a decoding tile are, against float64."""
from __future__ import annotations

import math

import pytest
import torch

import exact_attention_113_b200 as fa
from tests import paged_reference as ref
from tests.test_paged_gpu import Batch

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


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
