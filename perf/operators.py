"""The serving and training operators around paged attention: cases, plain forms and calls.

Four operators:

``plan``   one engine step's page tables: from the request lengths, the new tokens' positions and
           cache slots, the cumulative lengths and the block table grown from a free list.
``rope``   RMS norm of every query and key head, then the rotary position rotation; the serving
           form also writes K and V into the paged cache, the training form writes the layout the
           attention takes.
``rope_bwd``  its gradients: inputs and norm weights.
``attn``   attention of each request's new tokens over its paged cache (one token: decoding;
           many: a prefill chunk), causal to the end of the request, optional sliding window.

``own`` False: the definitions in elementary torch operations, fp32 (rounded once).
``own`` True: the same through exact_attention_113_b200.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoding step of a few requests: the smallest call of a step, all latency
        dict(name="plan_decode_8", op="plan", reqs=8, chunk=1, share=0.0, ctx=900, page=16, pad=0, mix=1),
        # a step that mixes decoding requests with prefill chunks, padded for a captured graph
        dict(name="plan_mixed_200", op="plan", reqs=200, chunk=300, share=0.15, ctx=5000, page=16, pad=77, mix=2),
        # a large batch of new prompts: many tokens, nothing in the cache yet
        dict(name="plan_prompts_1024", op="plan", reqs=1024, chunk=257, share=1.0, ctx=0, page=64, pad=0, mix=3),
        # decoding: one token of each of 33 requests, K and V go to the cache
        dict(name="rope_decode_33", op="rope", serve=True, batch=1, length=33, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, dtype="bf16", page=16, pages=600, mix=4),
        # a full prefill budget of 8192 tokens
        dict(name="rope_chunk_8192", op="rope", serve=True, batch=1, length=8192, heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, dtype="bf16", page=64, pages=300, mix=5),
        # a training batch, every head its own K and V, [B, H, L, D] out
        dict(name="rope_train_b4_l8192", op="rope", serve=False, batch=4, length=8192, heads=48, kv_heads=48, dim=64,
             rot=64, interleaved=False, dtype="fp16", page=0, pages=0, mix=6),
        # gradients of a short odd batch, pairs interleaved, half of each head rotated
        dict(name="rope_bwd_l1000", op="rope_bwd", serve=False, batch=1, length=1000, heads=12, kv_heads=12, dim=64,
             rot=32, interleaved=True, dtype="fp16", page=0, pages=0, mix=7),
        # gradients of a long training batch with shared K/V heads
        dict(name="rope_bwd_b2_l16384", op="rope_bwd", serve=False, batch=2, length=16384, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, dtype="bf16", page=0, pages=0, mix=8),
        # one request decoding over a short context: all latency
        dict(name="attn_decode_1", op="attn", reqs=1, chunk=1, share=0.0, ctx=1000, heads=32, kv_heads=8, dim=128,
             window=-1, dtype="bf16", page=16, mix=9),
        # a decoding batch with ragged contexts, bound by reading the cache
        dict(name="attn_decode_64", op="attn", reqs=64, chunk=1, share=0.0, ctx=12000, heads=32, kv_heads=8, dim=128,
             window=-1, dtype="bf16", page=16, mix=10),
        # decoding requests beside prefill chunks, sliding window, no shared heads
        dict(name="attn_mixed_20", op="attn", reqs=20, chunk=500, share=0.4, ctx=6000, heads=16, kv_heads=16, dim=64,
             window=4096, dtype="fp16", page=64, mix=11),
        # long prompts in chunks of up to 4096 tokens: bound by the matrix products
        dict(name="attn_prefill_2", op="attn", reqs=2, chunk=4096, share=1.0, ctx=12288, heads=32, kv_heads=8, dim=128,
             window=-1, dtype="bf16", page=128, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_bwd", "attn", "attn"])
    mix = rng.randrange(1 << 20)
    if op == "plan":
        reqs = _log(rng, 1, 1024)
        return dict(op=op, reqs=reqs, chunk=_log(rng, 1, 257), share=rng.choice([0.0, 0.1, 0.5, 1.0]),
                    ctx=rng.choice([0, _log(rng, 1, 8000)]), page=rng.choice([16, 32, 64, 128, 256]),
                    pad=rng.choice([0, rng.randrange(1, 200)]), mix=mix)
    heads, kv_heads = rng.choice([(32, 8), (48, 48), (12, 12), (16, 16), (16, 2), (14, 2), (8, 1)])
    dim = rng.choice([64, 128, rng.choice([16, 32, 48, 80, 96, 112])])
    dtype = rng.choice(["fp16", "bf16"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("rope", "rope_bwd"):
        serve = op == "rope" and rng.random() < 0.6
        # at most the elements of the largest listed case of the kind
        most = (8192 * 48 * 128 if serve else 32768 * 40 * 128) // ((heads + 2 * kv_heads) * dim)
        tokens = _log(rng, 1 if serve else 16, max(17, min(most, 32768)))
        batch = 1 if serve else rng.choice([1, 1, 2, 3])
        rot = dim if rng.random() < 0.7 else max(16, dim // 32 * 16)
        return dict(op=op, serve=serve, batch=batch, length=max(1, tokens // batch), heads=heads, kv_heads=kv_heads,
                    dim=dim, rot=rot, interleaved=rng.random() < 0.3, dtype=dtype, page=page if serve else 0,
                    pages=(2 * tokens + page) // page + 8 if serve else 0, mix=mix)
    window = rng.choice([-1, -1, _log(rng, 16, 4096)])
    if rng.random() < 0.5:  # decoding
        reqs = _log(rng, 1, 64)
        ctx = _log(rng, 1, max(2, min(16000, 12000 * 64 * 8 * 128 // (reqs * kv_heads * dim * 2))))
        return dict(op=op, reqs=reqs, chunk=1, share=0.0, ctx=ctx, heads=heads, kv_heads=kv_heads, dim=dim, window=window,
                    dtype=dtype, page=page, mix=mix)
    reqs = _log(rng, 1, 24)
    chunk = _log(rng, 2, max(3, min(4096, 8192 // reqs)))
    ctx = rng.choice([0, _log(rng, 1, max(2, min(12288, 32 * 2 * 4096 * 8000 // (heads * reqs * chunk))))])
    return dict(op=op, reqs=reqs, chunk=chunk, share=rng.choice([0.3, 1.0]), ctx=ctx, heads=heads, kv_heads=kv_heads,
                dim=dim, window=window, dtype=dtype, page=page, mix=mix)


def _lengths(case):
    """Ragged (new tokens, tokens in the cache) of every request: the case's shape, not its data."""
    r = random.Random(case["mix"])
    new, ctx = [], []
    for _ in range(case["reqs"]):
        long = case["chunk"] > 1 and r.random() < case["share"]
        new.append(r.randint(max(1, case["chunk"] // 2), case["chunk"]) if long else 1)
        ctx.append(r.randint(case["ctx"] // 3, case["ctx"]) if case["ctx"] else 0)
    if case["share"] >= 1.0 and case["chunk"] > 1:
        new[0] = case["chunk"]  # the longest chunk is there
    return new, ctx


def _pages(tokens, page):
    return -(-tokens // page)


def _visible(new, ctx, window):
    """Query-key pairs of one request and the keys any of its queries sees."""
    pairs = sum(min(ctx + i + 1, window + 1 if window >= 0 else 1 << 60) for i in range(new))
    return pairs, min(ctx + new, (window + new) if window >= 0 else 1 << 60)


def work(case):
    if case["op"] == "plan":
        new, ctx = _lengths(case)
        n, t = case["reqs"], sum(new) + case["pad"]
        grown = sum(_pages(c + q, case["page"]) - _pages(c, case["page"]) for q, c in zip(new, ctx))
        # lengths in; cumulative and total lengths, positions (4 B) and slots (8 B) out; new pages
        # read from the free list and written to the table; the partly filled page of a request read
        return {"bytes": 8 * n + 4 * (n + 1) + 4 * n + 12 * t + 8 * grown + 4 * n, "flops": 4 * t}
    if case["op"] in ("rope", "rope_bwd"):
        t = case["batch"] * case["length"]
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        table = 4 * case["rot"] * (t if case["serve"] else case["length"])
        if case["op"] == "rope_bwd":
            return {"bytes": 6 * t * (h + hk) * d + table + 4 * t, "flops": 16 * t * (h + hk) * d}
        rows = h + 2 * hk if case["serve"] else h + hk
        return {"bytes": 4 * t * rows * d + table + (12 if case["serve"] else 4) * t, "flops": 8 * t * (h + hk) * d}
    new, ctx = _lengths(case)
    pairs = keys = 0
    for q, c in zip(new, ctx):
        p, k = _visible(q, c, case["window"])
        pairs, keys = pairs + p, keys + k
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    return {"bytes": 4 * keys * hk * d + 4 * sum(new) * h * d + 4 * sum(new) * h, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ the inputs
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _table(case, new, ctx, g):
    """A block table whose rows hold the pages of the tokens in the cache (-1 behind them), and the
    free pages, all in random order."""
    page, n = case["page"], case["reqs"]
    have = torch.tensor([_pages(c, page) for c in ctx], device="cuda")
    need = torch.tensor([_pages(c + q, page) for q, c in zip(new, ctx)], device="cuda")
    width = int(need.max()) + 3
    total = int(need.sum()) + 5
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(width, device="cuda")
    held = at[None, :] < have[:, None]
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[held] = order[: int(have.sum())]
    return table, order[int(have.sum()):].contiguous(), total


def _cos_sin(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]])

    if case["op"] == "plan":
        new, ctx = _lengths(case)
        table, free, _ = _table(case, new, ctx, g)
        return dict(case=case, q_lens=_ints(new), ctx_lens=_ints(ctx), table=table, free=free, page=case["page"],
                    tokens=sum(new) + case["pad"])

    if case["op"] in ("rope", "rope_bwd"):
        b, n, h, hk, d = case["batch"], case["length"], case["heads"], case["kv_heads"], case["dim"]
        qkv = normal(b, n, h + 2 * hk, d)  # one projection's output: q, k, v side by side
        s = dict(case=case, q=qkv[:, :, :h], k=qkv[:, :, h:h + hk], v=qkv[:, :, h + hk:],
                 wq=1 + 0.1 * normal(d), wk=1 + 0.1 * normal(d))
        if case["serve"]:
            r = random.Random(case["mix"])
            far = 16384
            s["positions"] = _ints([[r.randrange(far) for _ in range(n)]])
            slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:n]
            if n > 4:  # padding at the end of a captured batch
                s["positions"][0, n - 2:] = -1
                slots[n - 2:] = -1
            s["slots"] = slots
            s["k_cache"] = normal(case["pages"], case["page"], hk, d)
            s["v_cache"] = normal(case["pages"], case["page"], hk, d)
            s["q_out"] = torch.zeros((b, n, h, d), dtype=qkv.dtype, device="cuda")
            s["cos_sin"] = _cos_sin(far, case["rot"])
        else:
            s["positions"] = torch.arange(n, dtype=torch.int32, device="cuda").expand(b, n)
            s["cos_sin"] = _cos_sin(n, case["rot"])
        if case["op"] == "rope_bwd":
            s["dq_out"] = normal(b, h, n, d).transpose(1, 2)  # the attention's gradients, [B, H, L, D]
            s["dk_out"] = normal(b, hk, n, d).transpose(1, 2)
        return s

    new, ctx = _lengths(case)
    table, free, total = _table(case, new, ctx, g)
    page = case["page"]
    have = torch.tensor([_pages(c, page) for c in ctx], device="cuda")
    need = torch.tensor([_pages(c + q, page) for q, c in zip(new, ctx)], device="cuda")
    at = torch.arange(table.shape[1], device="cuda")
    fresh = (at[None, :] >= have[:, None]) & (at[None, :] < need[:, None])
    table[fresh] = free[: int(fresh.sum())]
    starts = [0]
    for q in new:
        starts.append(starts[-1] + q)
    hk, d = case["kv_heads"], case["dim"]
    return dict(case=case, q=normal(starts[-1], case["heads"], d), k_cache=normal(total, page, hk, d),
                v_cache=normal(total, page, hk, d), table=table, cu_q=_ints(starts),
                kv_lens=_ints([c + q for q, c in zip(new, ctx)]), most_q=max(new), most_k=max(c + q for q, c in zip(new, ctx)))


# ------------------------------------------------------------------ plain forms
def _plan(s):
    page, tokens, table, free = s["page"], s["tokens"], s["table"], s["free"]
    q, ctx = s["q_lens"].long(), s["ctx_lens"].long()
    kv = ctx + q
    ends = torch.cumsum(q, 0)
    cu_q = torch.cat([ends.new_zeros(1), ends])
    have, need = (ctx + page - 1) // page, (kv + page - 1) // page
    grown = need - have
    first = torch.cumsum(grown, 0) - grown
    at = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (at >= have[:, None]) & (at < need[:, None])
    source = (first[:, None] + at - have[:, None]).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[source], table))
    t = torch.arange(tokens, device="cuda")
    row = torch.searchsorted(ends, t, right=True)
    real = row < q.numel()
    row = row.clamp(max=q.numel() - 1)
    pos = torch.where(real, ctx[row] + t - cu_q[row], -1)
    slot = table[row, pos.clamp(min=0) // page].long() * page + pos.clamp(min=0) % page
    return (cu_q.int(), kv.int(), pos.int(), torch.where(real, slot, -1), table,
            torch.stack([ends[-1], grown.sum(), grown.sum() * 0]).int())


def _turn(x, cos, sin, rot, interleaved, sign=1.0):
    """The rotation of the first `rot` values of each head by its position's angles."""
    a = x[..., 0:rot:2] if interleaved else x[..., : rot // 2]
    b = x[..., 1:rot:2] if interleaved else x[..., rot // 2:rot]
    c, s = cos[..., None, :], sin[..., None, :] * sign
    u, w = a * c - b * s, b * c + a * s
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _angles(s, f):
    rot = s["case"]["rot"]
    rows = s["cos_sin"][s["positions"].long().clamp(min=0)].to(f)
    return rows[..., : rot // 2], rows[..., rot // 2:], rot, s["case"]["interleaved"]


def _rope(s):
    cos, sin, rot, inter = _angles(s, torch.float32)

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        return _turn(y, cos, sin, rot, inter).to(w.dtype)

    q, k = one(s["q"], s["wq"]), one(s["k"], s["wk"])
    if not s["case"]["serve"]:
        return q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous()
    real = s["slots"] >= 0
    slots = s["slots"][real]
    s["q_out"][0, real] = q[0, real]
    s["k_cache"].flatten(0, 1)[slots] = k[0, real]
    s["v_cache"].flatten(0, 1)[slots] = s["v"][0, real]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _rope_bwd(s):
    cos, sin, rot, inter = _angles(s, torch.float32)

    def one(x, w, dy):
        x, g = x.float(), _turn(dy.float(), cos, sin, rot, inter, -1.0)
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r
        dw = (g * n).sum((0, 1, 2), dtype=torch.float64).float()
        g = g * w.float()
        return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(w.dtype), dw

    (dq, dwq), (dk, dwk) = one(s["q"], s["wq"], s["dq_out"]), one(s["k"], s["wk"], s["dk_out"])
    return dq, dk, dwq, dwk


def _attn(s):
    case, cu_q, kv = s["case"], s["cu_q"].long(), s["kv_lens"].long()
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    n, nq, nk = case["reqs"], s["most_q"], s["most_k"]
    lens = cu_q[1:] - cu_q[:-1]
    i = torch.arange(nq, device="cuda")
    j = torch.arange(nk, device="cuda")
    row = (cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float()  # [n, nq, h, d], padded
    pages = s["table"][:, : _pages(nk, page)].long().clamp(min=0)
    k, v = (c[pages].flatten(1, 2)[:, :nk].permute(0, 2, 1, 3).float() for c in (s["k_cache"], s["v_cache"]))
    q = q.view(n, nq, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, h // hk * nq, d)
    score = (q @ k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(n, hk, h // hk, nq, nk)
    at = (kv - lens)[:, None] + i  # a query's place in its request
    seen = (j[None, None] <= at[..., None]) & (j[None, None] < kv[:, None, None])
    if case["window"] >= 0:
        seen &= j[None, None] >= at[..., None] - case["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    out = (score.view(n, hk, h // hk * nq, nk) @ v).view(n, hk, h // hk, nq, d) / total.clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, nq, h, d)
    lse = lse.permute(0, 3, 1, 2).reshape(n, nq, h)
    real = i[None] < lens[:, None]
    return out[real].to(s["q"].dtype), lse[real]


def run(s):
    if own:
        return _own(s)
    return {"plan": _plan, "rope": _rope, "rope_bwd": _rope_bwd, "attn": _attn}[s["case"]["op"]](s)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import exact_attention_113_b200 as fa

    case = s["case"]
    if case["op"] == "plan":
        p = fa.paged_plan(s["q_lens"], s["ctx_lens"], s["table"], s["free"], s["page"], s["tokens"])
        return p.cu_q, p.kv_lens, p.positions, p.slots, s["table"], p.counts
    if case["op"] == "attn":
        return fa.flash_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"], s["kv_lens"], causal=True,
                                  window_left=case["window"])
    b, n, h, hk, d = case["batch"], case["length"], case["heads"], case["kv_heads"], case["dim"]
    same = dict(eps=EPS, interleaved=case["interleaved"])
    if case["op"] == "rope_bwd":
        return fa.qk_norm_rope_bwd(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], s["positions"], s["dq_out"],
                                   s["dk_out"], **same)
    if case["serve"]:
        fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], s["positions"], q_out=s["q_out"], v=s["v"],
                        k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"], **same)
        return s["q_out"], s["k_cache"], s["v_cache"]
    q = torch.empty((b, h, n, d), dtype=s["q"].dtype, device="cuda")
    k = torch.empty((b, hk, n, d), dtype=s["q"].dtype, device="cuda")
    fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], s["positions"], q_out=q.transpose(1, 2),
                    k_out=k.transpose(1, 2), **same)
    return q, k


# ------------------------------------------------------------------ 64 bits
def _exact_rotated(x, w, s):
    """RMS norm and rotation in float64, the rotation as a complex product."""
    case = s["case"]
    rot, x = case["rot"], x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    rows = s["cos_sin"].double()[s["positions"].long().clamp(min=0)]
    turn = torch.complex(rows[..., : rot // 2], rows[..., rot // 2:]).unsqueeze(-2)
    head = y[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
    head = head if case["interleaved"] else head.transpose(-1, -2)
    z = torch.view_as_real(torch.complex(head[..., 0], head[..., 1]) * turn)
    z = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        q, k = _exact_rotated(s["q"], s["wq"].double(), s), _exact_rotated(s["k"], s["wk"].double(), s)
        if not case["serve"]:
            return q.permute(0, 2, 1, 3).contiguous(), k.permute(0, 2, 1, 3).contiguous()
        out, kc, vc = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
        keep = (s["slots"] >= 0).nonzero().flatten()
        page, place = s["slots"][keep] // case["page"], s["slots"][keep] % case["page"]
        out[0, keep], kc[page, place], vc[page, place] = q[0, keep], k[0, keep], s["v"][0, keep].double()
        return out, kc, vc
    if case["op"] == "rope_bwd":
        grads = []
        for x, w, dy in ((s["q"], s["wq"], s["dq_out"]), (s["k"], s["wk"], s["dk_out"])):
            x, w = x.double().requires_grad_(), w.double().requires_grad_()
            grads.append(torch.autograd.grad(_exact_rotated(x, w, s), (x, w), dy.double()))
        return grads[0][0], grads[1][0], grads[0][1], grads[1][1]
    outs, lses = [], []
    cu, kv = s["cu_q"].tolist(), s["kv_lens"].tolist()
    group, scale = case["heads"] // case["kv_heads"], 1 / math.sqrt(case["dim"])
    for b in range(case["reqs"]):
        q = s["q"][cu[b]:cu[b + 1]].double()
        pages = s["table"][b, : _pages(kv[b], case["page"])].long()
        k, v = (c[pages].reshape(-1, case["kv_heads"], case["dim"])[: kv[b]].double() for c in (s["k_cache"], s["v_cache"]))
        at = torch.arange(kv[b] - q.shape[0], kv[b], device="cuda")[:, None]
        gap = at - torch.arange(kv[b], device="cuda")[None]
        hidden = gap < 0 if case["window"] < 0 else (gap < 0) | (gap > case["window"])
        o, e = [], []
        for h in range(case["heads"]):
            x = torch.einsum("qd,kd->qk", q[:, h], k[:, h // group]) * scale
            x = x.masked_fill(hidden, -math.inf)
            e.append(torch.logsumexp(x, -1))
            o.append(torch.softmax(x, -1) @ v[:, h // group])
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(e, 1))
    return torch.cat(outs), torch.cat(lses)
