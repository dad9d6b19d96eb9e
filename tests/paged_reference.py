"""64-bit references of the serving operators, request by request, and the
rounding bounds their GPU tests use.  Shares no code with the package."""
from __future__ import annotations

import math

import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def attention(q, k_cache, v_cache, table, cu_q, kv_lens, scale, causal, wl, wr):
    """(out, lse, abs) in float64: abs is sum_j p_j |v_j|, and, for fp16's
    smallest weights, the sum of |v_j| over the visible keys."""
    page = k_cache.shape[1]
    H, H_kv = q.shape[1], k_cache.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag, total = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    cu, kv = cu_q.tolist(), kv_lens.tolist()
    for b in range(len(kv)):
        n, m = cu[b + 1] - cu[b], kv[b]
        if n <= 0 or m <= 0:
            continue
        pages = table[b, : -(-m // page)].long()
        k, v = (c[pages].flatten(0, 1)[:m].double() for c in (k_cache, v_cache))
        x = torch.arange(m - n, m, device=q.device)[:, None]
        j = torch.arange(m, device=q.device)[None]
        seen = torch.ones((n, m), dtype=torch.bool, device=q.device)
        if causal:
            seen &= j <= x
        if wr >= 0:
            seen &= j <= x + wr
        if wl >= 0:
            seen &= j >= x - wl
        any_seen = seen.any(1)
        for h in range(H):
            g = h // (H // H_kv)
            s = (q[cu[b]:cu[b + 1], h].double() @ k[:, g].T * scale).masked_fill(~seen, -math.inf)
            top = s.amax(1, keepdim=True).masked_fill(~any_seen[:, None], 0.0)
            e = (s - top).exp()
            l = e.sum(1, keepdim=True).clamp(min=1e-300)
            p = e / l
            rows = slice(cu[b], cu[b + 1])
            out[rows, h] = p @ v[:, g]
            mag[rows, h] = p @ v[:, g].abs()
            total[rows, h] = seen.double() @ v[:, g].abs()
            lse[rows, h] = torch.where(any_seen, top[:, 0] + l[:, 0].log(), -math.inf)
    return out, lse, mag, total


def attention_bound(out, mag, total, dtype):
    """|error| of the kernel's O: P and O are rounded to 16 bits once each
    (half a step of each term, of the result); a fp32 score of up to 128
    products is off by at most 128 * 2^-24 * scale * sum |q k|, about 2^-14
    here, which enters a weight and the normaliser once each (2^-13 of mag);
    fp16 weights below 2^-14 keep an absolute step of 2^-24."""
    h = HALF[dtype]
    b = h * (1 + 2.0 ** -6) * (out.abs() + mag) + 2.0 ** -13 * mag
    if dtype == torch.float16:
        b = b + 2.0 ** -25 * total + 2.0 ** -25
    return b


LSE_BOUND = 2.0 ** -12   # 2^-14 of the score, fp32 sums of some thousand terms, ex2 and lg2


def turn(y, cos_sin, positions, rot, interleaved, sign=1.0):
    y = y.clone()
    rows = cos_sin.double()[positions.long().clamp(min=0)]
    c, s = rows[..., None, : rot // 2], rows[..., None, rot // 2:] * sign
    if interleaved:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., : rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., : rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def norm_rope(x, w, cos_sin, positions, eps, interleaved):
    """The operator's definition in float64; differentiable in x and w."""
    y = x
    if w is not None:
        y = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w
    return turn(y, cos_sin, positions, cos_sin.shape[1], interleaved)


def norm_rope_bound(x, w, cos_sin, positions, eps, interleaved, y, dtype):
    """Half a step of the result, and fp32: about ten roundings of 2^-24 of
    values no larger than the row's largest normed value."""
    z = x
    if w is not None:
        z = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w
    top = 2 * z.abs().amax(-1, keepdim=True)
    return HALF[dtype] * (1 + 2.0 ** -10) * y.abs() + 2.0 ** -19 * top + 2.0 ** -25


def plan(q_lens, ctx_lens, table, free, page, num_tokens):
    """Plain integers, one token at a time."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    taken, cu, kv, pos, slots, missing = 0, [0], [], [], [], 0
    for b, (q, c) in enumerate(zip(q_lens, ctx_lens)):
        q, c = max(q, 0), max(c, 0)
        have, need = -(-c // page), min(-(-(c + q) // page), width)
        for i in range(have, need):
            table[b][i] = free[taken] if taken < len(free) else -1
            taken += 1
        lost = 0
        for x in range(c, c + q):
            pg = table[b][x // page] if x // page < width else -1
            pos.append(x)
            slots.append(pg * page + x % page if pg >= 0 else -1)
            lost += pg < 0 and x // page >= have or x // page >= width
        missing += lost
        cu.append(cu[-1] + q)
        kv.append(c + q)
    counts = [cu[-1], min(taken, len(free)), missing]
    pad = max(0, num_tokens - len(pos))
    return (cu, kv, (pos + [-1] * pad)[:num_tokens], (slots + [-1] * pad)[:num_tokens], table, counts)
