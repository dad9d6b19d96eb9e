"""fa_qk_norm_rope and its gradient against float64 (tests/paged_reference)."""
from __future__ import annotations

import pytest
import torch

import exact_attention_113_b200 as fa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _inputs(shape, H, H_kv, D, rot, dtype, seed=0, far=4000, weights=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s):
        return torch.randn(s, generator=g, device="cuda")

    qkv = n(*shape, H + 2 * H_kv, D).to(dtype)
    q, k, v = qkv.split([H, H_kv, H_kv], dim=-2)
    w = [(1 + 0.2 * n(D)).to(dtype) if weights else None for _ in range(2)]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * f
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, far, shape, generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, w[0], w[1], cos_sin, pos


def _want(x, w, cos_sin, pos, inter):
    x, w = x.double(), None if w is None else w.double()
    y = ref.norm_rope(x, w, cos_sin, pos, EPS, inter)
    return y, x, w


def _assert_rows(got, x, w, cos_sin, pos, inter):
    y, xd, wd = _want(x, w, cos_sin, pos, inter)
    b = ref.norm_rope_bound(xd, wd, cos_sin, pos, EPS, inter, y, got.dtype)
    assert ((got.double() - y).abs() <= b).all()


@pytest.mark.parametrize("D,rot", [(16, 16), (32, 16), (48, 48), (64, 64), (64, 32), (80, 80),
                                   (96, 64), (112, 112), (128, 128), (128, 0)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
def test_forward(D, rot, dtype, inter):
    q, k, v, wq, wk, cs, pos = _inputs((37,), 7, 3, D, rot, dtype, seed=D + rot)
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, interleaved=inter)
    _assert_rows(qo, q, wq, cs, pos, inter)
    _assert_rows(ko, k, wk, cs, pos, inter)


@pytest.mark.parametrize("T,H,H_kv", [(1, 1, 1), (1, 32, 8), (5, 1, 0), (300, 48, 48), (64, 128, 1)])
def test_head_layouts(T, H, H_kv):
    q, k, v, wq, wk, cs, pos = _inputs((T,), H, H_kv, 64, 64, torch.bfloat16, seed=T)
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, cs, pos.long(), eps=EPS)
    _assert_rows(qo, q, wq, cs, pos, False)
    if H_kv:
        _assert_rows(ko, k, wk, cs, pos, False)


def test_batched_strided_and_broadcast_positions():
    B, L, H, H_kv, D = 3, 50, 6, 2, 64
    q, k, v, wq, wk, cs, _ = _inputs((B, L), H, H_kv, D, D, torch.float16, seed=3)
    pos = torch.arange(7, 7 + L, device="cuda").expand(B, L)
    qo = torch.empty(B, H, L, D, dtype=q.dtype, device="cuda")
    ko = torch.empty(B, H_kv, L, D, dtype=q.dtype, device="cuda")
    fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, q_out=qo.transpose(1, 2), k_out=ko.transpose(1, 2))
    _assert_rows(qo.transpose(1, 2), q, wq, cs, pos, False)
    _assert_rows(ko.transpose(1, 2), k, wk, cs, pos, False)


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_and_without_norm(inter):
    q, k, v, wq, _, cs, pos = _inputs((40,), 5, 2, 128, 64, torch.bfloat16, seed=4)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    fa.qk_norm_rope(q, k, wq, None, cs, pos, eps=EPS, interleaved=inter, q_out=q, k_out=k)
    _assert_rows(q, q0, wq, cs, pos, inter)
    _assert_rows(k, k0, None, cs, pos, inter)
    assert torch.equal(v, v0)


def test_zero_rows_with_zero_eps_are_not_touched_by_others():
    # a row of zeros and eps > 0: zeros out; extreme rows stay finite in fp32
    q, k, v, wq, wk, cs, pos = _inputs((9,), 4, 2, 64, 64, torch.bfloat16, seed=5)
    q = q.clone()
    q[3] = 0
    q[4] *= 1e15
    q[5] *= 1e-12
    qo, _ = fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS)
    assert (qo[3] == 0).all()
    _assert_rows(qo, q, wq, cs, pos, False)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("D,page", [(128, 16), (80, 64), (16, 1)])
def test_cache_write(heads_first, D, page):
    T, H, H_kv, pages = 45, 8, 3, 60 // page + 2
    q, k, v, wq, wk, cs, pos = _inputs((T,), H, H_kv, D, D, torch.float16, seed=6)
    pos = pos.clone()
    pos[4], pos[-1], pos[6] = -1, -1, cs.shape[0]      # padding: nothing of it is written
    g = torch.Generator(device="cuda").manual_seed(7)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    slots[-1] = -1
    slots[9], slots[10] = -1, pages * page             # q_out yes, cache no
    shape = (pages, H_kv, page, D) if heads_first else (pages, page, H_kv, D)
    caches = [torch.full(shape, 7.0, dtype=q.dtype, device="cuda") for _ in range(2)]
    kc, vc = (c.transpose(1, 2) if heads_first else c for c in caches)
    qo = torch.full_like(q.contiguous(), 5.0)
    ko = torch.full_like(k.contiguous(), 5.0)
    fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, q_out=qo, k_out=ko, v=v, k_cache=kc, v_cache=vc,
                    slots=slots)
    real = (pos >= 0) & (pos < cs.shape[0])
    assert (qo[~real] == 5).all() and (ko[~real] == 5).all()
    _assert_rows(qo[real], q[real], wq, cs, pos[real], False)
    _assert_rows(ko[real], k[real], wk, cs, pos[real], False)
    kept = real & (slots >= 0) & (slots < pages * page)
    pg, row = slots[kept] // page, slots[kept] % page
    assert torch.equal(kc[pg, row], ko[kept]) and torch.equal(vc[pg, row], v[kept])
    touched = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    touched[pg, row] = True
    assert (kc[~touched] == 7).all() and (vc[~touched] == 7).all()


def test_padding_rows_may_hold_nan():
    q, k, v, wq, wk, cs, pos = _inputs((6,), 4, 2, 64, 64, torch.float16, seed=8)
    q, k, pos = q.clone(), k.clone(), pos.clone()
    q[2], k[2], pos[2] = float("nan"), float("nan"), -1
    real = pos >= 0
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS)
    _assert_rows(qo[real], q[real], wq, cs, pos[real], False)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, q, k, eps=EPS)
    assert (dq[2] == 0).all() and (dk[2] == 0).all()
    assert torch.isfinite(dwq).all() and torch.isfinite(dwk).all()


# ------------------------------------------------------------------ gradient
def _reference_grads(x, w, cs, pos, inter, dy):
    x = x.double().requires_grad_()
    wd = None if w is None else w.double().requires_grad_()
    y = ref.norm_rope(x, wd, cs, pos, EPS, inter)
    ins = (x,) if wd is None else (x, wd)
    g = torch.autograd.grad(y, ins, dy.double())
    return g[0], (g[1] if wd is not None else None)


def _grad_bounds(x, w, cs, pos, inter, dy, dx, dtype):
    """dx: half a step, and some twenty fp32 roundings of terms of at most
    r * (|w g| + |x r| mean |w g x r|).  dw: chains of at most 2^6 fp32 sums
    and two more levels, of sum |g x r|."""
    x, g = x.double(), ref.turn(dy.double(), cs, pos, cs.shape[1], inter, -1.0)
    if w is None:
        return ref.HALF[dtype] * dx.abs() * (1 + 2.0 ** -10) + 2.0 ** -20 * g.abs().amax(-1, keepdim=True) \
            + 2.0 ** -25, None
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n, wg = x * r, g * w.double()
    top = r * (wg.abs().amax(-1, keepdim=True)
               + n.abs().amax(-1, keepdim=True) * (wg * n).abs().mean(-1, keepdim=True))
    bx = ref.HALF[dtype] * dx.abs() * (1 + 2.0 ** -10) + 2.0 ** -18 * top + 2.0 ** -25
    bw = 2.0 ** -17 * (g * n).abs().flatten(0, -2).sum(0) + 2.0 ** -40
    return bx, bw


@pytest.mark.parametrize("D,rot,shape,H,H_kv", [
    (64, 64, (1,), 1, 1), (128, 128, (70,), 8, 2), (64, 32, (2, 33), 5, 5), (112, 16, (40,), 3, 1),
    (16, 16, (2, 100), 4, 2), (48, 48, (500,), 7, 1), (128, 128, (3000,), 32, 8), (32, 32, (9,), 64, 0),
])
@pytest.mark.parametrize("dtype,inter", [(torch.float16, False), (torch.bfloat16, True)])
def test_backward(D, rot, shape, H, H_kv, dtype, inter):
    q, k, v, wq, wk, cs, pos = _inputs(shape, H, H_kv, D, rot, dtype, seed=D + H)
    g = torch.Generator(device="cuda").manual_seed(99)
    # the layout of an attention gradient, [.., H, L, D] seen as [.., L, H, D]
    def grad(t):
        s = (*t.shape[:-3], t.shape[-2], t.shape[-3], t.shape[-1])
        return torch.randn(s, generator=g, device="cuda").to(dtype).transpose(-3, -2)
    dyq, dyk = grad(q), grad(k)
    got = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, dyq, dyk, eps=EPS, interleaved=inter)
    again = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, dyq, dyk, eps=EPS, interleaved=inter)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    for x, w, dy, dx, dw in ((q, wq, dyq, got[0], got[2]), (k, wk, dyk, got[1], got[3])):
        if x.shape[-2] == 0:
            assert (dw == 0).all()
            continue
        wx, ww = _reference_grads(x, w, cs, pos, inter, dy)
        bx, bw = _grad_bounds(x, w, cs, pos, inter, dy, wx, dtype)
        assert ((dx.double() - wx).abs() <= bx).all()
        assert ((dw.double() - ww).abs() <= bw).all()


def test_backward_against_differences():
    q, k, v, wq, wk, cs, pos = _inputs((12,), 3, 1, 64, 32, torch.float16, seed=21)
    g = torch.Generator(device="cuda").manual_seed(5)
    dyq = torch.randn(q.shape, generator=g, device="cuda").half()
    dyk = torch.randn(k.shape, generator=g, device="cuda").half()
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, dyq, dyk, eps=EPS)
    for x, w, dy, dx, dw in ((q, wq, dyq, dq, dwq), (k, wk, dyk, dk, dwk)):
        x, w, dy = x.double(), w.double(), dy.double()
        dirx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        dirw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)

        def f(t):
            return (ref.norm_rope(x + t * dirx, w + t * dirw, cs, pos, EPS, False) * dy).sum()
        h = 1e-5
        slope = (f(h) - f(-h)) / (2 * h)
        mine = (dx.double() * dirx).sum() + (dw.double() * dirw).sum()
        wx, ww = _reference_grads(x, w, cs, pos, False, dy)
        bx, bw = _grad_bounds(x, w, cs, pos, False, dy, wx, torch.float16)
        bound = (bx * dirx.abs()).sum() + (bw * dirw.abs()).sum()
        # differences of step h are off by h^2 times a third derivative
        assert (slope - mine).abs() <= bound + 1e-4


def test_backward_without_norm_in_place_and_padding():
    q, k, v, _, wk, cs, pos = _inputs((30,), 4, 2, 64, 64, torch.bfloat16, seed=22)
    pos = pos.clone()
    pos[7] = -1
    g = torch.Generator(device="cuda").manual_seed(6)
    dyq = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    dyk = torch.randn(k.shape, generator=g, device="cuda").bfloat16()
    y0 = dyq.clone()
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, None, wk, cs, pos, dyq, dyk, eps=EPS, dq=dyq)
    assert dq.data_ptr() == dyq.data_ptr() and dwq is None
    real = pos >= 0
    want = ref.turn(y0.double(), cs, pos, 64, False, -1.0)
    b = ref.HALF[torch.bfloat16] * want.abs() * (1 + 2.0 ** -10) + 2.0 ** -18
    assert ((dq.double() - want).abs() <= b)[real].all() and (dq[7] == 0).all() and (dk[7] == 0).all()
    wx, ww = _reference_grads(k[real], wk, cs, pos[real], False, dyk[real])
    bx, bw = _grad_bounds(k[real], wk, cs, pos[real], False, dyk[real], wx, torch.bfloat16)
    assert ((dk[real].double() - wx).abs() <= bx).all() and ((dwk.double() - ww).abs() <= bw).all()


def test_backward_of_no_tokens():
    q, k, v, wq, wk, cs, pos = _inputs((0,), 4, 2, 64, 64, torch.bfloat16)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, q, k)
    assert dq.numel() == 0 and (dwq == 0).all() and (dwk == 0).all()


def test_other_stream_and_graph():
    q, k, v, wq, wk, cs, pos = _inputs((64,), 8, 2, 128, 128, torch.bfloat16, seed=30)
    q, k = q.contiguous(), k.contiguous()
    s = torch.cuda.Stream()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, q_out=qo, k_out=ko)
        s.synchronize()
    _assert_rows(qo, q, wq, cs, pos, False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.qk_norm_rope(q, k, wq, wk, cs, pos, eps=EPS, q_out=qo, k_out=ko)
        grads = fa.qk_norm_rope_bwd(q, k, wq, wk, cs, pos, qo, ko, eps=EPS)
    q.copy_(torch.randn_like(q))
    pos.copy_(pos.flip(0))
    g.replay()
    torch.cuda.synchronize()
    _assert_rows(qo, q, wq, cs, pos, False)
    wx, ww = _reference_grads(q, wq, cs, pos, False, qo)
    bx, bw = _grad_bounds(q, wq, cs, pos, False, qo, wx, q.dtype)
    assert ((grads[0].double() - wx).abs() <= bx).all() and ((grads[2].double() - ww).abs() <= bw).all()
