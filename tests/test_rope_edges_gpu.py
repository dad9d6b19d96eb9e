"""fa_qk_norm_rope and its gradient without an epsilon, with axes of one element,
and where a warp takes many steps, against float64."""
from __future__ import annotations

import pytest
import torch

import exact_attention_113_b200 as fa
from tests import paged_reference as ref
from tests.test_rope_gpu import EPS, _inputs

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def _rows_ok(got, x, w, cos_sin, pos, inter, eps=EPS):
    x, w = x.double(), None if w is None else w.double()
    y = ref.norm_rope(x, w, cos_sin, pos, eps, inter)
    bound = ref.norm_rope_bound(x, w, cos_sin, pos, eps, inter, y, got.dtype)
    assert ((got.double() - y).abs() <= bound).all()


def _grads(x, w, cs, pos, inter, dy, eps):
    """The gradients by differentiation, and their bounds.  dx: half a step of
    the result, and some twenty fp32 roundings of terms of at most r (|w g| +
    |x r| mean |w g x r|), 2^-18 of them.  dw: fp32 sums along a lane's rows
    (a few hundred here at most, each off by 2^-24 of the sum so far: 2^-16)
    and two short levels above."""
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    dx, dw = torch.autograd.grad(ref.norm_rope(xd, wd, cs, pos, eps, inter), (xd, wd), dy.double())
    x, w = x.double(), w.double()
    g = ref.turn(dy.double(), cs, pos, cs.shape[1], inter, -1.0)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n, wg = x * r, g * w
    top = r * (wg.abs().amax(-1, keepdim=True)
               + n.abs().amax(-1, keepdim=True) * (wg * n).abs().mean(-1, keepdim=True))
    bx = ref.HALF[dy.dtype] * dx.abs() * (1 + 2.0 ** -10) + 2.0 ** -18 * top + 2.0 ** -25
    bw = 2.0 ** -15 * (g * n).abs().flatten(0, -2).sum(0) + 2.0 ** -40
    return dx, dw, bx, bw


def _backward_ok(q, k, wq, wk, cs, pos, dyq, dyk, got, inter, eps):
    for x, w, dy, dx, dw in ((q, wq, dyq, got[0], got[2]), (k, wk, dyk, got[1], got[3])):
        wx, ww, bx, bw = _grads(x, w, cs, pos, inter, dy, eps)
        assert ((dx.double() - wx).abs() <= bx).all()
        assert ((dw.double() - ww).abs() <= bw).all()


# ------------------------------------------------------------ no epsilon
# heads that do not fill a warp's step (4 rows at D 128, 8 at 64, 32 at 16)
@pytest.mark.parametrize("D,H,H_kv", [(128, 8, 2), (64, 12, 3), (16, 3, 1), (48, 9, 5), (64, 8, 8)])
@pytest.mark.parametrize("dtype,inter", [(F16, True), (BF16, False)])
def test_zero_epsilon(D, H, H_kv, dtype, inter):
    q, k, _, wq, wk, cs, pos = _inputs((50,), H, H_kv, D, D, dtype, seed=D)
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=0.0, interleaved=inter)
    _rows_ok(qo, q, wq, cs, pos, inter, 0.0)
    _rows_ok(ko, k, wk, cs, pos, inter, 0.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    dyq, dyk = (torch.randn(x.shape, generator=g, device="cuda").to(dtype) for x in (q, k))
    got = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, dyq, dyk, eps=0.0, interleaved=inter)
    _backward_ok(q, k, wq, wk, cs, pos, dyq, dyk, got, inter, 0.0)


def test_rows_of_zeros_without_an_epsilon():
    q, k, _, wq, wk, cs, pos = _inputs((9,), 5, 2, 64, 64, BF16, seed=4)
    q = q.clone()
    q[3] = 0
    qo, _ = fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=0.0)
    assert (qo[3] == 0).all()
    keep = torch.arange(9, device="cuda") != 3
    _rows_ok(qo[keep], q[keep], wq, cs, pos[keep], False, 0.0)
    got = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, torch.zeros_like(q), k, eps=0.0)
    assert (got[0] == 0).all() and (got[2] == 0).all()


# ------------------------------------------------------------ axes of one element
def _odd(x, axes):
    """x with strides of 3 elements along its one-element axes."""
    for a in axes:
        assert x.shape[a] == 1
    stride = [3 if a in axes else n for a, n in enumerate(x.stride())]
    return x.as_strided(x.shape, stride, x.storage_offset())


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("shape,H,H_kv,axes", [((50,), 1, 1, (1,)), ((1, 1), 6, 2, (0, 1)),
                                               ((1, 40), 1, 1, (0, 2))])
def test_strides_of_one_element_axes(D, shape, H, H_kv, axes):
    q, k, v, wq, wk, cs, pos = _inputs(shape, H, H_kv, D, D, BF16, seed=D)
    q, k, v = (_odd(x.contiguous(), axes) for x in (q, k, v))
    qo, ko = (_odd(torch.full(x.shape, 5.0, dtype=BF16, device="cuda"), axes) for x in (q, k))
    T = pos.numel()
    cache = [torch.full((T // 16 + 1, 16, H_kv, D), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
    fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, q_out=qo, k_out=ko, v=v, k_cache=cache[0],
                    v_cache=cache[1], slots=torch.arange(T, device="cuda"))
    _rows_ok(qo, q, wq, cs, pos, False)
    _rows_ok(ko, k, wk, cs, pos, False)
    assert torch.equal(cache[0].flatten(0, 1)[:T], ko.reshape(T, H_kv, D))
    assert torch.equal(cache[1].flatten(0, 1)[:T], v.reshape(T, H_kv, D))
    dyq, dyk = _odd(q.clone(), axes), _odd(k.clone(), axes)
    got = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, dyq, dyk, eps=EPS,
                              dq=_odd(torch.empty_like(q.contiguous()), axes))
    _backward_ok(q, k, wq, wk, cs, pos, dyq, dyk, got, False, EPS)


# ------------------------------------------------------------ many steps a warp
# On 148 SMs, with a cache, the query rows of a token are chunks of 8, 6, 2, 4 and
# 5 steps, the last one some rows short (without a cache two of them are cut), and
# a warp walks 10 to 40 steps, so that every place of its ring is used again.
@pytest.mark.parametrize("T,H,H_kv,D,rot,dtype,inter", [
    (6000, 30, 6, 128, 128, BF16, False),
    (9000, 44, 12, 64, 32, F16, True),
    (1500, 47, 7, 128, 64, F16, True),      # chunks of 2 steps: a token's rows over several warps
    (9000, 50, 18, 32, 32, BF16, False),
    (5000, 130, 70, 16, 16, F16, False),
])
@pytest.mark.parametrize("cached", [False, True])
def test_long_walks(T, H, H_kv, D, rot, dtype, inter, cached):
    q, k, v, wq, wk, cs, pos = _inputs((T,), H, H_kv, D, rot, dtype, seed=T + D)
    g = torch.Generator(device="cuda").manual_seed(2)
    pos = pos.long()
    pos[torch.randperm(T, generator=g, device="cuda")[: T // 9]] = -1        # padding in between
    pos[T // 2: T // 2 + 300] = -1
    pos[7], pos[T - 1] = cs.shape[0], 1 << 40
    real = (pos >= 0) & (pos < cs.shape[0])
    qo, ko = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    kw = {}
    if cached:
        page = 16
        slots = torch.randperm(T + 200, generator=g, device="cuda")[:T]
        slots[::13] = -1
        caches = [torch.full((T // page + 14, page, H_kv, D), 7.0, dtype=dtype, device="cuda")
                  for _ in range(2)]
        kw = dict(v=v, k_cache=caches[0], v_cache=caches[1], slots=slots)
    fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, interleaved=inter, q_out=qo, k_out=ko, **kw)
    _rows_ok(qo[real], q[real], wq, cs, pos[real], inter)
    _rows_ok(ko[real], k[real], wk, cs, pos[real], inter)
    assert (qo[~real] == 5).all() and (ko[~real] == 5).all()
    if cached:
        kept = real & (slots >= 0)
        for cache, rows in zip(caches, (ko, v)):
            want = torch.full_like(cache, 7.0)
            want.flatten(0, 1)[slots[kept]] = rows[kept]
            assert torch.equal(cache, want)


@pytest.mark.parametrize("wide", [False, True])
def test_long_walks_to_heads_first(wide):
    B, L, H, H_kv, D = 3, 2500, 22, 6, 64
    q, k, _, wq, wk, cs, pos = _inputs((B, L), H, H_kv, D, D, BF16, seed=77)
    pos = pos.long() if wide else pos
    pos[1, 100:200], pos[2, -1] = -1, -3
    qo = torch.full((B, H, L, D), 5.0, dtype=BF16, device="cuda")
    ko = torch.full((B, H_kv, L, D), 5.0, dtype=BF16, device="cuda")
    fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, q_out=qo.transpose(1, 2), k_out=ko.transpose(1, 2))
    real = pos >= 0
    for out, x, w in ((qo.transpose(1, 2), q, wq), (ko.transpose(1, 2), k, wk)):
        _rows_ok(out[real], x[real], w, cs, pos[real], False)
        assert (out[~real] == 5).all()


@pytest.mark.parametrize("T,H,H_kv,D", [(6000, 30, 6, 128), (9000, 20, 12, 64)])
def test_long_backward(T, H, H_kv, D):
    q, k, _, wq, wk, cs, pos = _inputs((T,), H, H_kv, D, D, BF16, seed=T)
    g = torch.Generator(device="cuda").manual_seed(3)
    dyq, dyk = (torch.randn(x.shape, generator=g, device="cuda").bfloat16() for x in (q, k))
    got = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, dyq, dyk, eps=EPS)
    _backward_ok(q, k, wq, wk, cs, pos, dyq, dyk, got, False, EPS)
