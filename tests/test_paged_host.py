"""Host-side checks of the serving entries (no kernel is launched): the status
codes of the C entries and the refusals of the torch wrappers."""
import ctypes

import pytest
import torch

import exact_attention_113_b200 as fa
from exact_attention_113_b200 import binding
from exact_attention_113_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return fa.load()


# ------------------------------------------------------------ fa_fwd_paged
GOOD = dict(q=16, qt=512, qh=64, k=16, v=16, cp=4096, ct=128, ch=64, table=16, ts=8, cu=16, kv=16,
            out=16, ot=512, oh=64, lse=0, T=8, B=2, H=8, H_kv=2, D=64, pages=32, page=32, maxp=8,
            scale=0.125, causal=1, wl=-1, wr=-1, dtype=0, ws=256, wsb=None)


def _paged(**kw):
    a = dict(GOOD)
    a.update(kw)
    wsb = fa.fa_paged_workspace_bytes(a["D"]) if a["wsb"] is None else a["wsb"]
    return fa.fa_fwd_paged(a["q"], a["qt"], a["qh"], a["k"], a["v"], a["cp"], a["ct"], a["ch"],
                           a["table"], a["ts"], a["cu"], a["kv"], a["out"], a["ot"], a["oh"],
                           a["lse"], a["T"], a["B"], a["H"], a["H_kv"], a["D"], a["pages"],
                           a["page"], a["maxp"], a["scale"], a["causal"], a["wl"], a["wr"],
                           a["dtype"], a["ws"], wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(B=0), -2), (dict(H=0), -2), (dict(H_kv=3), -2), (dict(pages=0), -2),
    (dict(maxp=0), -2), (dict(H=129, H_kv=1), -2), (dict(T=(1 << 30) + 1), -2),
    (dict(D=40), -3), (dict(D=144), -3), (dict(D=8), -3), (dict(dtype=2), -4), (dict(dtype=-1), -4),
    (dict(page=8), -6), (dict(page=48), -6), (dict(page=192), -6), (dict(page=0), -6),
    (dict(scale=-1.0), -6), (dict(scale=float("nan")), -6), (dict(ts=7), -6),
    (dict(q=0), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(table=0), -1), (dict(cu=0), -1),
    (dict(kv=0), -1), (dict(out=0), -1), (dict(ws=0), -1),
    (dict(q=8), -5), (dict(k=24), -5), (dict(out=4), -5), (dict(lse=2), -5), (dict(ws=128), -5),
    (dict(table=2), -5), (dict(qt=510), -5), (dict(qh=0), -5), (dict(ct=-64), -5), (dict(ch=4), -5),
    (dict(cp=1), -5), (dict(ot=4), -5), (dict(wsb=1024), -9),
])
def test_paged_argument_errors(lib, kw, code):
    assert _paged(**kw) == code


def test_paged_empty_is_a_no_op(lib):
    assert _paged(T=0) == 0
    assert _paged(T=0, q=0, out=0, k=0, ws=0) == 0


def test_paged_workspace_bytes(lib):
    # two tiles of 256 rows of D fp32 and a float2, and a counter, for each SM
    sms = 148
    assert fa.fa_paged_workspace_bytes(64) == sms * (2 * 256 * (64 * 4 + 8) + 8)
    assert fa.fa_paged_workspace_bytes(40) == 0


# ------------------------------------------------------------ fa_paged_plan
PLAN = dict(q=16, ctx=16, table=16, ts=8, free=16, n_free=4, B=2, maxp=8, page=16, T=8, cu=16, kv=16,
            pos=16, slots=16, counts=16)


def _plan(**kw):
    a = dict(PLAN)
    a.update(kw)
    return fa.fa_paged_plan(a["q"], a["ctx"], a["table"], a["ts"], a["free"], a["n_free"], a["B"],
                            a["maxp"], a["page"], a["T"], a["cu"], a["kv"], a["pos"], a["slots"],
                            a["counts"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -2), (dict(n_free=-1), -2), (dict(maxp=-1), -2), (dict(T=-1), -2),
    (dict(page=0), -6), (dict(ts=7), -6), (dict(q=0), -1), (dict(ctx=0), -1), (dict(table=0), -1),
    (dict(free=0), -1), (dict(cu=0), -1), (dict(kv=0), -1), (dict(pos=0), -1), (dict(slots=0), -1),
    (dict(counts=0), -1), (dict(q=2), -5), (dict(slots=4), -5),
])
def test_plan_argument_errors(lib, kw, code):
    assert _plan(**kw) == code


# ------------------------------------------------------------ fa_qk_norm_rope
def _args(**kw):
    a = binding.FaRopeArgs()
    for n in ("q", "k", "v", "q_out", "k_out"):
        setattr(a, n, binding.FaRows(16, 4096, 512, 64))
    base = dict(q_weight=16, k_weight=16, cos_sin=16, positions=16, positions_stride_b=8,
                positions_stride_l=1, B=2, L=8, H=8, H_kv=2, D=64, rot_dim=64, max_pos=32,
                dtype=0, eps=1e-6)
    base.update(kw)
    for n, x in base.items():
        setattr(a, n, x)
    return a


R0 = binding.FaRows(0, 4096, 512, 64)
BAD = binding.FaRows(8, 4096, 512, 64)
ODD = binding.FaRows(16, 4096, 513, 64)
CACHE = dict(k_cache=16, v_cache=16, cache_stride_page=4096, cache_stride_token=128,
             cache_stride_head=64, num_pages=4, page_size=32, slots=16)

COMMON = [
    (dict(B=0), -2), (dict(L=-1), -2), (dict(H=0), -2), (dict(H_kv=-1), -2), (dict(B=1 << 30), -2),
    (dict(D=40), -3), (dict(D=256), -3), (dict(dtype=2), -4), (dict(rot_dim=8), -6),
    (dict(rot_dim=80), -6), (dict(rot_dim=-16), -6), (dict(max_pos=-1), -6), (dict(eps=-1.0), -6),
    (dict(eps=float("nan")), -6), (dict(positions_64=2), -6), (dict(q=R0), -1), (dict(k=R0), -1),
    (dict(q_out=R0), -1), (dict(k_out=R0), -1), (dict(positions=0), -1), (dict(cos_sin=0), -1),
    (dict(q=BAD), -5), (dict(k_out=ODD), -5), (dict(q_weight=8), -5), (dict(cos_sin=4), -5),
    (dict(positions=2), -5), (dict(positions=4, positions_64=1), -5),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(CACHE, k_cache=0), -1), (dict(CACHE, v_cache=0), -1), (dict(CACHE, v=R0), -1),
    (dict(CACHE, slots=0), -1), (dict(CACHE, num_pages=0), -6), (dict(CACHE, page_size=0), -6),
    (dict(CACHE, slots=4), -5), (dict(CACHE, cache_stride_head=4), -5), (dict(CACHE, k_cache=8), -5),
])
def test_rope_argument_errors(lib, kw, code):
    assert fa.fa_qk_norm_rope(_args(**kw), None) == code


def _bwd(ws=256, wsb=None, dq=R0, dk=R0, dwq=16, dwk=16, **kw):
    ok = binding.FaRows(16, 4096, 512, 64)
    dq, dk = (ok if x is R0 else x for x in (dq, dk))
    wsb = fa.fa_qk_norm_rope_bwd_workspace_bytes(64) if wsb is None else wsb
    return fa.fa_qk_norm_rope_bwd(_args(**kw), dq, dk, dwq, dwk, ws, wsb, None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dwq=0), -1), (dict(dwk=0), -1), (dict(q_weight=0), -1), (dict(dq=BAD), -5),
    (dict(dk=binding.FaRows(0, 1, 1, 1)), -1), (dict(dwq=2), -5), (dict(ws=0), -1), (dict(ws=64), -5),
    (dict(wsb=16), -9),
])
def test_rope_bwd_argument_errors(lib, kw, code):
    assert _bwd(**kw) == code


def test_rope_null_and_empty(lib):
    null = ctypes.POINTER(binding.FaRopeArgs)()
    assert fa.load().fa_qk_norm_rope(null, None) == -1
    assert fa.fa_qk_norm_rope(_args(L=0, q=R0, k=R0, q_out=R0, k_out=R0, positions=0), None) == 0


# ------------------------------------------------------------ torch wrappers
def test_wrappers_refuse_bad_tensors(lib):
    i32 = torch.int32
    q = torch.zeros(4, 8, 64, dtype=torch.float16)
    k = torch.zeros(4, 2, 64, dtype=torch.float16)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    table, cu, kv = torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError):
        fa.flash_fwd_paged(q, cache, cache, table, cu, kv)                      # CPU tensors
    with pytest.raises(ValueError):
        fa.flash_fwd_paged(q[None], cache, cache, table, cu, kv)                # not 3-D
    with pytest.raises(TypeError):
        fa.flash_fwd_paged(q.float(), cache.float(), cache.float(), table, cu, kv)
    with pytest.raises(TypeError):
        fa.flash_fwd_paged(q, cache.bfloat16(), cache.bfloat16(), table, cu, kv)
    with pytest.raises(ValueError):
        fa.flash_fwd_paged(q, cache, cache[:2], table, cu, kv)                  # caches differ
    with pytest.raises(ValueError):
        fa.flash_fwd_paged(q, cache, cache, table, cu[:2], kv)                  # cu_q too short
    with pytest.raises(ValueError):
        fa.flash_fwd_paged(q, cache, cache, table.long(), cu, kv)
    with pytest.raises(ValueError):
        fa.flash_fwd_paged(q, cache.transpose(2, 3), cache.transpose(2, 3), table, cu, kv)
    w, cs, pos = torch.ones(64, dtype=q.dtype), torch.zeros(9, 64), torch.zeros(4, dtype=i32)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, k, w, w, cs, pos)                                    # CPU tensors
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, k[:2], w, w, cs, pos)                                # token axes differ
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, k, w.float(), w, cs, pos)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, k, w, w, cs.half(), pos)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, k, w, w, cs, pos.float())
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q, k, w, w, cs, pos, k_cache=cache)                     # half a cache
    with pytest.raises(TypeError):
        fa.qk_norm_rope(q.double(), k.double(), None, None, cs, pos)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_bwd(q, k, w, w, cs, pos, q[:2], k)
    with pytest.raises(ValueError):
        fa.paged_plan(kv, kv, table, kv, 16, 8)                                 # CPU tensors
    with pytest.raises(ValueError):
        fa.paged_plan(kv.long(), kv, table, kv, 16, 8)
    with pytest.raises(ValueError):
        fa.paged_plan(kv, kv, table[:1], kv, 16, 8)


@pytest.mark.parametrize("kw", [
    dict(kv="ctx"), dict(kv="q"), dict(cu="ctx"), dict(pos="slots"), dict(counts="cu"),
    dict(table="free"), dict(slots="table"),
])
def test_plan_refuses_overlap(lib, kw):
    # every array on a page of its own but one, which shares its last bytes
    names = ("q", "ctx", "table", "free", "cu", "kv", "pos", "slots", "counts")
    at = {n: 4096 * (i + 1) for i, n in enumerate(names)}
    for a, b in kw.items():
        at[a] = at[b]
    assert _plan(**at) == -6
