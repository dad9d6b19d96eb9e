"""Workspaces that own less memory than they have elements are refused before
anything is launched."""
import pytest
import torch

import exact_attention_113_b200 as fa
from exact_attention_113_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return fa.load()


def _bad(device):
    """One byte seen as many, and every other byte."""
    n = 1 << 26
    return (torch.zeros(1, dtype=torch.uint8, device=device).expand(n),
            torch.zeros(2 * n, dtype=torch.uint8, device=device)[::2])


def test_serving_entries():
    i32 = torch.int32
    q = torch.zeros(4, 8, 64, dtype=torch.float16)
    k = torch.zeros(4, 2, 64, dtype=torch.float16)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    table, cu, kv = torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    w, cs, pos = torch.ones(64, dtype=q.dtype), torch.zeros(9, 64), torch.zeros(4, dtype=i32)
    for ws in _bad("cpu"):
        with pytest.raises(ValueError, match="contiguous"):
            fa.flash_fwd_paged(q, cache, cache, table, cu, kv, workspace=ws)
        with pytest.raises(ValueError, match="contiguous"):
            fa.qk_norm_rope_bwd(q, k, w, w, cs, pos, q, k, workspace=ws)


@pytest.mark.gpu
def test_training_and_decoding_entries():
    q = torch.zeros(1, 2, 64, 64, dtype=torch.float16, device="cuda")
    lse = torch.zeros(1, 2, 64, device="cuda")
    f8 = q.to(torch.float8_e4m3fn)
    host = q.cpu()
    for ws in _bad("cuda"):
        for call in (lambda: fa.flash_fwd(q, q, q, n_splits=2, workspace=ws),
                     lambda: fa.flash_fwd_fp8(f8, f8, f8, n_splits=2, workspace=ws),
                     lambda: fa.flash_bwd(q, q, q, q, q, lse, workspace=ws),
                     lambda: fa.flash_bwd(q, q, q, q, q, lse, workspace=ws,
                                          mask=torch.ones(1, 1, 64, 64, dtype=torch.bool, device="cuda")),
                     lambda: fa.flash_fwd_host(host, host, host, workspace=ws)):
            with pytest.raises(ValueError, match="contiguous"):
                call()
    torch.cuda.synchronize()
