"""fa_fwd_paged against float64 (tests/paged_reference), and the serving
operators run together as a step of an engine runs them."""
from __future__ import annotations

import math

import pytest
import torch

import exact_attention_113_b200 as fa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


class Batch:
    """Ragged requests over a paged cache, its pages in random order.  Whatever
    no query sees is NaN: page tails, unused pages, unused table entries name
    a page full of NaN."""

    def __init__(self, q_lens, kv_lens, H, H_kv, D, dtype, page, seed=0, heads_first=False,
                 pad_rows=3, std=1.0, first_seen=None):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def n(*s):
            return (std * torch.randn(s, generator=g, device="cuda")).to(dtype)

        B = len(q_lens)
        self.q_lens = q_lens
        used = [-(-m // page) for m in kv_lens]
        self.pages = sum(used) + 3
        order = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)
        nan_page = int(order[-1])
        width = max(used + [1]) + 2
        self.table = torch.full((B, width), nan_page, dtype=torch.int32, device="cuda")
        shape = (self.pages, H_kv, page, D) if heads_first else (self.pages, page, H_kv, D)
        self.k, self.v = (torch.full(shape, math.nan, dtype=dtype, device="cuda") for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        at = 0
        for b, m in enumerate(kv_lens):
            pg = order[at:at + used[b]]
            at += used[b]
            self.table[b, : used[b]] = pg
            for c in (self.k, self.v):
                x = torch.full((used[b] * page, H_kv, D), math.nan, dtype=dtype, device="cuda")
                x[:m] = n(m, H_kv, D)
                if first_seen is not None:
                    x[: first_seen[b]] = math.nan
                c[pg.long()] = x.view(used[b], page, H_kv, D)
        cu = [0]
        for x in q_lens:
            cu.append(cu[-1] + x)
        self.T = cu[-1] + pad_rows
        self.q = n(self.T, H, D)
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.kv_lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        out = torch.full_like(self.q, 3.0)
        lse = torch.full(self.q.shape[:2], 5.0, dtype=torch.float32, device="cuda")
        fa.flash_fwd_paged(self.q, self.k, self.v, self.table, self.cu_q, self.kv_lens, out=out,
                           lse=lse, **kw)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == 0
        return out, lse

    def check(self, out, lse, causal=True, wl=-1, wr=-1, scale=None):
        scale = 1 / math.sqrt(self.q.shape[2]) if scale is None else scale
        clean = [torch.nan_to_num(c, nan=0.0) for c in (self.k, self.v)]
        want, wlse, mag, total = ref.attention(self.q, *clean, self.table, self.cu_q, self.kv_lens,
                                               scale, causal, wl, wr)
        real = int(self.cu_q[-1])
        err = (out.double() - want).abs()[:real]
        bound = ref.attention_bound(want, mag, total, self.q.dtype)[:real]
        assert torch.isfinite(out[:real].float()).all()
        assert (err <= bound).all(), float((err - bound).max())
        seen = torch.isfinite(wlse[:real])
        assert torch.equal(torch.isneginf(lse[:real]), ~seen)
        assert (out[:real][~seen] == 0).all()
        assert ((lse[:real].double() - wlse[:real])[seen].abs() <= ref.LSE_BOUND).all()
        assert (out[real:] == 3).all() and (lse[real:] == 5).all()   # rows no request owns


RAGGED = ([1, 5, 0, 130, 300, 2, 1], [1, 700, 40, 130, 1200, 129, 128])


@pytest.mark.parametrize("H,H_kv,D,page,dtype", [
    (4, 4, 64, 16, F16), (8, 2, 128, 16, BF16), (7, 1, 64, 32, F16), (6, 2, 128, 64, F16),
    (16, 1, 32, 128, BF16), (2, 2, 16, 256, F16), (5, 1, 48, 16, BF16), (4, 2, 80, 32, F16),
    (3, 3, 96, 16, F16), (8, 1, 112, 16, BF16), (128, 1, 128, 16, BF16), (70, 1, 64, 16, F16),
])
def test_ragged_requests(H, H_kv, D, page, dtype):
    b = Batch(*RAGGED, H, H_kv, D, dtype, page, seed=D + page)
    b.check(*b.run())


@pytest.mark.parametrize("kw", [
    dict(causal=True, window_left=0), dict(causal=True, window_left=100),
    dict(causal=True, window_left=127), dict(causal=False), dict(causal=False, window_right=70),
    dict(causal=False, window_left=33, window_right=5),
    dict(causal=True, window_left=(1 << 31) - 1, window_right=9),
])
@pytest.mark.parametrize("D,H,H_kv", [(64, 4, 4), (128, 8, 2)])
def test_windows(kw, D, H, H_kv):
    b = Batch(*RAGGED, H, H_kv, D, F16, 16, seed=5)
    wr = kw.get("window_right", -1)
    b.check(*b.run(**kw), causal=kw["causal"], wl=kw.get("window_left", -1), wr=wr)


def test_rows_without_keys():
    # fewer tokens in the cache than new ones: the first rows see nothing
    b = Batch([5, 3, 200, 1], [3, 0, 20, 0], 4, 2, 64, F16, 16)
    b.check(*b.run())
    b.check(*b.run(causal=False, window_left=4), causal=False, wl=4)


def test_all_requests_empty():
    b = Batch([0, 0], [10, 0], 4, 2, 64, F16, 16)
    out, lse = b.run()
    assert (out == 3).all() and (lse == 5).all()


@pytest.mark.parametrize("H,H_kv,D,n,m,dtype", [
    (8, 8, 128, 1, 9000, BF16), (16, 1, 64, 1, 40000, F16), (32, 8, 128, 1, 20000, BF16),
    (4, 1, 128, 2, 60000, F16), (8, 1, 64, 1500, 5000, BF16),
])
def test_one_long_request_is_cut_over_all_ctas(H, H_kv, D, n, m, dtype):
    b = Batch([n], [m], H, H_kv, D, dtype, 16, seed=m)
    out, lse = b.run()
    b.check(out, lse)
    again = b.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("n", [1, 3, 150, 400, 1000])
def test_many_requests(n):
    g = torch.Generator().manual_seed(n)
    kv = torch.randint(1, 500, (n,), generator=g).tolist()
    b = Batch([1] * n, kv, 4, 2, 64, BF16, 16, seed=n)
    b.check(*b.run())


def test_evicted_pages_before_the_window():
    # pages wholly before every query's window are gone (-1 or another
    # request's); the tokens before it in the first visible page hold NaN
    q, kv, wl = [1, 40, 1], [1000, 900, 333], 256
    first = [max(0, m - n - wl) for n, m in zip(q, kv)]
    b = Batch(q, kv, 4, 2, 64, F16, 16, seed=9, first_seen=first)
    for r, f in enumerate(first):
        b.table[r, : f // 16] = -1 if r else b.pages + 5
    want = Batch(q, kv, 4, 2, 64, F16, 16, seed=9, first_seen=first)
    out, lse = b.run(window_left=wl)
    want.check(out, lse, wl=wl)


def test_heads_first_cache_strided_q_and_out():
    H, H_kv, D = 8, 2, 128
    b = Batch(*RAGGED, H, H_kv, D, BF16, 32, seed=11, heads_first=True)
    wide = torch.randn(b.T, H + 2 * H_kv, D, device="cuda").to(BF16)   # a projection's output
    wide[:, :H] = b.q
    q = wide[:, :H]
    store = torch.full((H, b.T, D + 8), 3.0, dtype=BF16, device="cuda")
    out = store[..., :D].transpose(0, 1)
    lse = torch.full((b.T, H), 5.0, dtype=torch.float32, device="cuda")
    fa.flash_fwd_paged(q, b.k, b.v, b.table[:, :], b.cu_q, b.kv_lens, out=out, lse=lse)
    b.check(out, lse)
    assert (store[..., D:] == 3).all()
    o2, none = fa.flash_fwd_paged(q, b.k, b.v, b.table, b.cu_q, b.kv_lens, return_lse=False)
    assert none is None and torch.equal(o2[: int(b.cu_q[-1])], out[: int(b.cu_q[-1])])


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (1.0, 3.0), (0.125, 30.0)])
def test_scales(scale, std):
    # large scores: the softmax is close to one key; q, k of 30 make scores of 10^4
    b = Batch([1, 70], [300, 500], 4, 2, 64, BF16, 16, seed=12, std=std)
    out, lse = b.run(scale=scale)
    if std == 1.0:
        b.check(out, lse, scale=scale)
        return
    clean = [torch.nan_to_num(c, nan=0.0) for c in (b.k, b.v)]
    want, wlse, mag, _ = ref.attention(b.q, *clean, b.table, b.cu_q, b.kv_lens, scale, True, -1, -1)
    real = int(b.cu_q[-1])
    # a score s is off by at most 2^-14 (see the bound) at |q k| terms of 1;
    # the terms here are std^2 * scale * 8 times as large
    off = 2.0 ** -14 * max(1.0, std * std * scale * 8)
    bound = ref.HALF[BF16] * 1.02 * (want.abs() + mag) + 2 * off * mag
    assert ((out.double() - want).abs() <= bound)[:real].all()
    assert ((lse.double() - wlse).abs() <= ref.LSE_BOUND + off + 2.0 ** -22 * wlse.abs())[:real].all()


def test_growing_maxima_rescale():
    # keys whose scores rise with the position: every block raises the row
    # maxima by far more than the threshold of the lazy rescale
    m, D = 1500, 64
    b = Batch([1, 200], [m, m], 4, 2, D, F16, 16, seed=13)
    ramp = torch.arange(m, device="cuda").to(torch.float32) / m
    for r in range(2):
        pg = b.table[r, : -(-m // 16)].long()
        k = b.k[pg].flatten(0, 1)
        k[:m] = (ramp[:, None, None] * 4).half()
        b.k[pg] = k.view(-1, 16, 2, D)
    b.q.fill_(2.0)       # scores 2 * 4 * ramp * 64 / 8 = 64 * ramp
    b.check(*b.run())


def test_offsets_past_32_bits():
    # page strides that put the used pages beyond 2^31 elements
    H, H_kv, D, page = 4, 1, 128, 16
    b = Batch([1, 40], [500, 900], H, H_kv, D, BF16, page, seed=14)
    stride = (1 << 31) // b.pages // 8 * 8 + (1 << 20)
    big = [torch.zeros(stride * b.pages, dtype=BF16, device="cuda") for _ in range(2)]
    views = [t.as_strided((b.pages, page, H_kv, D), (stride, D, D, 1)) for t in big]
    for view, c in zip(views, (b.k, b.v)):
        view.copy_(c)
    assert (b.pages - 1) * stride > 1 << 31
    b.k, b.v = views
    b.check(*b.run())


def test_other_streams_at_once():
    s = [torch.cuda.Stream() for _ in range(2)]
    bs = [Batch([1] * 40, [700] * 40, 8, 2, 128, BF16, 16, seed=20 + i) for i in range(2)]
    torch.cuda.synchronize()
    got = []
    for st, b in zip(s, bs):
        with torch.cuda.stream(st):
            got.append([fa.flash_fwd_paged(b.q, b.k, b.v, b.table, b.cu_q, b.kv_lens)
                        for _ in range(4)][-1])
    torch.cuda.synchronize()
    for b, (out, lse) in zip(bs, got):
        real = int(b.cu_q[-1])
        o, e = out.clone(), lse.clone()
        o[real:], e[real:] = 3, 5
        b.check(o, e)


def test_graph_replay_with_other_lengths_and_pages():
    b = Batch([1, 5, 0, 130], [1, 700, 40, 130], 8, 2, 64, F16, 16, seed=30, pad_rows=300)
    b2 = Batch([3, 1, 60, 9], [80, 500, 300, 400], 8, 2, 64, F16, 16, seed=31, pad_rows=300)
    T, pages = max(b.T, b2.T), max(b.pages, b2.pages)
    width = max(b.table.shape[1], b2.table.shape[1])
    q = torch.zeros(T, 8, 64, dtype=F16, device="cuda")
    k, v = (torch.zeros(pages, 16, 2, 64, dtype=F16, device="cuda") for _ in range(2))
    table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    cu, kv = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(T, 8, dtype=torch.float32, device="cuda")
    ws = torch.empty(fa.fa_paged_workspace_bytes(64), dtype=torch.uint8, device="cuda")

    def put(x):
        q.zero_()
        q[: x.T] = x.q
        for dst, src in ((k, x.k), (v, x.v)):
            dst[: x.pages] = src
        table.fill_(-1)
        table[:, : x.table.shape[1]] = x.table
        cu.copy_(x.cu_q)
        kv.copy_(x.kv_lens)
        out.fill_(3)
        lse.fill_(5)

    def call():
        fa.flash_fwd_paged(q, k, v, table, cu, kv, out=out, lse=lse, workspace=ws)

    put(b)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in (b2, b):
        put(x)
        g.replay()
        torch.cuda.synchronize()
        x.check(out[: x.T], lse[: x.T])
        assert (out[x.T:] == 3).all()


def test_bad_lengths_are_cut():
    # cu_q beyond total_q, kv_len beyond the table: no access outside, the
    # other requests' rows as always
    b = Batch([2, 4, 3], [50, 60, 70], 4, 2, 64, F16, 16, seed=40, pad_rows=0)
    good, _ = b.run()
    b.cu_q[3] = 1000
    b.kv_lens[2] = 100000
    out, _ = b.run()
    assert torch.equal(out[:6], good[:6])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,page,wl", [(BF16, 16, -1), (F16, 64, 90)])
def test_serving_steps(dtype, page, wl):
    """Three requests served in steps (prefill in chunks, then decoding, in one
    captured-size batch), against the training path on the whole sequences."""
    H, H_kv, D, B = 8, 2, 64, 3
    lengths = [[150, 40, 1, 1, 1], [7, 0, 1, 1, 0], [1, 300, 0, 1, 1]]   # new tokens by step
    total = [sum(x) for x in lengths]
    g = torch.Generator(device="cuda").manual_seed(50)
    far = 600
    f = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * f
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    seqs = [torch.randn(n, H + 2 * H_kv, D, generator=g, device="cuda").to(dtype) for n in total]
    pages = sum(-(-n // page) for n in total) + 1
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    kc = torch.full((pages, page, H_kv, D), math.nan, dtype=dtype, device="cuda")
    vc = kc.clone()
    table = torch.full((B, far // page + 1), -1, dtype=torch.int32, device="cuda")
    T = max(sum(x[s] for x in lengths) for s in range(5)) + 2
    done, taken = [0] * B, 0
    outs = [[] for _ in range(B)]
    for s in range(5):
        new = [x[s] for x in lengths]
        p = fa.paged_plan(torch.tensor(new, dtype=torch.int32, device="cuda"),
                          torch.tensor(done, dtype=torch.int32, device="cuda"), table,
                          free[taken:].contiguous(), page, T)
        qkv = torch.full((T, H + 2 * H_kv, D), math.nan, dtype=dtype, device="cuda")
        at = 0
        for b in range(B):
            qkv[at:at + new[b]] = seqs[b][done[b]:done[b] + new[b]]
            at += new[b]
        q, k, v = qkv.split([H, H_kv, H_kv], dim=1)
        qo, _ = fa.qk_norm_rope(q, k, w[0], w[1], cs, p.positions, v=v, k_cache=kc, v_cache=vc,
                                slots=p.slots)
        out, _ = fa.flash_fwd_paged(qo, kc, vc, table, p.cu_q, p.kv_lens, window_left=wl)
        assert p.counts.tolist()[2] == 0
        taken += int(p.counts[1])
        at = 0
        for b in range(B):
            outs[b].append(out[at:at + new[b]])
            at += new[b]
            done[b] += new[b]
    assert fa.fa_get_device_status() == 0
    for b in range(B):
        q, k, v = (x[None] for x in seqs[b].split([H, H_kv, H_kv], dim=1))
        pos = torch.arange(total[b], device="cuda")[None]
        qo = torch.empty(1, H, total[b], D, dtype=dtype, device="cuda")
        ko = torch.empty(1, H_kv, total[b], D, dtype=dtype, device="cuda")
        fa.qk_norm_rope(q, k, w[0], w[1], cs, pos, q_out=qo.transpose(1, 2), k_out=ko.transpose(1, 2))
        vt = v.transpose(1, 2).contiguous()
        got = torch.cat(outs[b]).double()
        # the cache's k are the training path's, bit for bit; so one reference
        one = torch.arange(1, device="cuda", dtype=torch.int32)[None]
        cu = torch.tensor([0, total[b]], dtype=torch.int32, device="cuda")
        want, _, mag, tot = ref.attention(qo[0].transpose(0, 1), ko[0].transpose(0, 1)[None],
                                          vt[0].transpose(0, 1)[None], one, cu, cu[1:],
                                          1 / math.sqrt(D), True, wl, -1)
        assert ((got - want).abs() <= ref.attention_bound(want, mag, tot, dtype)).all()
        train, _ = fa.flash_fwd(qo, ko, vt, causal=True, window_left=wl)
        assert ((train[0].transpose(0, 1).double() - got).abs()
                <= 2 * ref.attention_bound(want, mag, tot, dtype)).all()


def test_given_stream_owns_what_is_allocated():
    # memory of another stream's pool could be in use there when this call runs
    def stream_of(t):
        for seg in torch.cuda.memory_snapshot():
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                return seg["stream"]

    b = Batch([1] * 3, [300] * 3, 8, 2, 128, BF16, 16, seed=40)
    cs, pos = torch.rand(400, 128, device="cuda"), (b.kv_lens - 1).repeat(b.T)[: b.T]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = fa.flash_fwd_paged(b.q, b.k, b.v, b.table, b.cu_q, b.kv_lens, stream=st)
    q2, k2 = fa.qk_norm_rope(b.q, b.q[:, :2], None, None, cs, pos, stream=st)
    w = torch.ones(128, dtype=BF16, device="cuda")
    grads = fa.qk_norm_rope_bwd(b.q, b.q[:, :2], w, w, cs, pos, b.q, b.q[:, :2], stream=st)
    plan = fa.paged_plan(b.kv_lens, b.kv_lens.clone(), b.table.clone(), b.kv_lens.clone(), 16, 9,
                         stream=st)
    for t in (out, lse, q2, k2, *grads, *plan):
        assert stream_of(t) == st.cuda_stream
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    st.synchronize()


@pytest.mark.parametrize("H,H_kv,q_lens", [
    (8, 1, [1, 2, 1]), (4, 2, [4, 5, 3]), (2, 2, [8, 9, 7]), (9, 1, [1, 1, 2]), (6, 1, [1, 260, 2]),
    (16, 1, [1, 9, 1]),
])
@pytest.mark.parametrize("D,wl", [(64, -1), (128, -1), (48, 200), (128, 90)])
def test_few_rows(H, H_kv, q_lens, D, wl):
    # up to 8 rows (tokens x heads of a group) four lanes share a row; around it
    b = Batch(q_lens, [777, 1030, 128], H, H_kv, D, BF16, 16, seed=H + D)
    b.check(*b.run(window_left=wl), wl=wl)


@pytest.mark.parametrize("wl", [-1, 300])
def test_growing_maxima_wide_heads(wl):
    # as above for D 128, where a masked block's exponentials are tried against
    # the old reference first (the products' sums of equal terms are exact)
    m, D = 1500, 128
    b = Batch([1, 200, 300], [m, m, 300], 4, 2, D, F16, 16, seed=13)
    for r, n in enumerate((m, m, 300)):
        pg = b.table[r, : -(-n // 16)].long()
        k = b.k[pg].flatten(0, 1)
        ramp = torch.arange(n, device="cuda").to(torch.float32) / n
        k[:n] = (ramp[:, None, None] * 2).half()
        b.k[pg] = k.view(-1, 16, 2, D)
    b.q.fill_(2.0)       # scores 2 * 2 * ramp * 128 / 11.3 = 45 * ramp
    b.check(*b.run(window_left=wl), wl=wl)


def test_requests_on_many_short_pieces():
    # decoding, verifying a few tokens and chunks side by side, more items than
    # blocks of the device: cuts fall on borders, inside items and near their ends
    g = torch.Generator().manual_seed(3)
    q = [1, 4, 33, 129, 257, 2, 64] * 30
    kv = [n + int(x) for n, x in zip(q, torch.randint(0, 900, (len(q),), generator=g))]
    b = Batch(q, kv, 8, 2, 128, BF16, 16, seed=41)
    out, lse = b.run()
    b.check(out, lse)
    again = b.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_graphs_and_eager_calls_share_a_workspace_in_turn():
    b = Batch([1, 300, 5, 1], [9000, 2000, 700, 50], 8, 2, 128, BF16, 16, seed=2)
    ws = torch.full((fa.fa_paged_workspace_bytes(128),), 255, dtype=torch.uint8, device="cuda")
    first, first_lse = b.run(workspace=ws)
    b.check(first, first_lse)
    args = (b.q, b.k, b.v, b.table, b.cu_q, b.kv_lens)
    out, lse = torch.empty_like(b.q), torch.empty_like(first_lse)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            fa.flash_fwd_paged(*args, out=out, lse=lse, workspace=ws)
    real = int(b.cu_q[-1])
    for i in range(6):
        if i == 3:
            ws.random_(0, 255)   # what another user of the memory leaves
        graphs[i % 2].replay()
        fa.flash_fwd_paged(*args, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(out[:real], first[:real]) and torch.equal(lse[:real], first_lse[:real])


def test_requests_share_pages():
    # one prompt's full pages at the head of the others' tables
    b = Batch([1, 200, 1, 3], [700, 640, 900, 500], 8, 2, 128, BF16, 64, seed=51)
    for r in (1, 2, 3):
        b.table[r, :7] = b.table[0, :7]
    b.check(*b.run())
    b.check(*b.run(window_left=222), wl=222)
