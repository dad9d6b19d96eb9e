"""fa_qk_norm_rope and its gradient without an epsilon, and with axes of one
element, against float64."""
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
