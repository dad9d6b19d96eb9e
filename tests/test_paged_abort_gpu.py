"""fa_fwd_paged's own abort path on the GPU, without a fault, through the
watchdog test library (see test_watchdog_abort_gpu.py): CTA 0 withholds the copy
of one block of K or V, the wait for it runs out after 10 ms, every role leaves
its loop, copies in flight land, and the launch ends with the timeout status.
The call is a captured one, whose every run has the same number in the
workspace's tickets: the next run gives the right rows only if the run that gave
up has counted its parts."""
from __future__ import annotations

import ctypes
import os
import time

import pytest
import torch

import exact_attention_113_b200 as fa
from exact_attention_113_b200 import build as fa_build
from tests.test_paged_gpu import Batch

pytestmark = pytest.mark.gpu
FA_OK, FA_ERR_TIMEOUT = 0, -8
F16 = torch.float16
V = 1 << 16     # 65536 + n: V's n-th block


@pytest.fixture(scope="module")
def hooks():
    if not os.path.exists(fa_build.TESTHOOKS_PATH) or fa_build.is_stale(fa_build.TESTHOOKS_PATH):
        fa_build.build(testhooks=True)
    lib = ctypes.CDLL(fa_build.TESTHOOKS_PATH)
    lib.fa_fwd_paged.argtypes = fa.load().fa_fwd_paged.argtypes
    lib.fa_fwd_paged.restype = ctypes.c_int
    lib.fa_get_device_status.argtypes = [ctypes.c_void_p]
    lib.fa_get_device_status.restype = ctypes.c_int
    lib.fa_test_set_withhold.argtypes = [ctypes.c_int]
    lib.fa_test_set_withhold.restype = ctypes.c_int
    yield lib
    lib.fa_test_set_withhold(-1)


class Call:
    def __init__(self, lib, b, ws):
        self.lib, self.b, self.ws = lib, b, ws
        self.out = torch.full_like(b.q, 3.0)
        self.lse = torch.full(b.q.shape[:2], 5.0, dtype=torch.float32, device="cuda")

    def __call__(self):
        b, (T, H, D) = self.b, self.b.q.shape
        pages, page, H_kv, _ = b.k.shape
        st = self.lib.fa_fwd_paged(
            b.q.data_ptr(), b.q.stride(0), b.q.stride(1), b.k.data_ptr(), b.v.data_ptr(),
            b.k.stride(0), b.k.stride(1), b.k.stride(2), b.table.data_ptr(), b.table.stride(0),
            b.cu_q.data_ptr(), b.kv_lens.data_ptr(), self.out.data_ptr(), self.out.stride(0),
            self.out.stride(1), self.lse.data_ptr(), T, b.kv_lens.numel(), H, H_kv, D, pages, page,
            b.table.shape[1], D ** -0.5, 1, -1, -1, fa.FA_F16, self.ws.data_ptr(), self.ws.numel(),
            torch.cuda.current_stream().cuda_stream)
        assert st == FA_OK

    def check(self):
        torch.cuda.synchronize()
        self.b.check(self.out, self.lse)
        self.out.fill_(3.0)
        self.lse.fill_(5.0)


CASES = {
    # one decoding request, cut over every CTA: CTA 0 has the item's first part
    "decode": lambda D: Batch([1], [200000], 8, 1, D, F16, 64, seed=90),
    # chunks: pairs of tiles, items cut between two CTAs, ragged first and last blocks
    "chunks": lambda D: Batch([1500, 700], [2000, 900], 8, 2, D, F16, 16, seed=91),
    # more items than CTAs: whole ones behind each other
    "many": lambda D: Batch([1, 40, 3, 1] * 60, [900, 500, 333, 700] * 60, 8, 2, D, F16, 16, seed=92),
}


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("name", list(CASES))
def test_withheld_copy_ends_the_launch_and_the_next_run_is_right(hooks, name, D):
    b = CASES[name](D)
    ws = torch.zeros(fa.fa_paged_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    call = Call(hooks, b, ws)
    assert hooks.fa_get_device_status(None) == FA_OK       # nothing pending
    call()
    call.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for withheld in (0, 2, V, V + 1, V + 2):
        assert hooks.fa_test_set_withhold(withheld) == FA_OK
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        g.replay()
        assert hooks.fa_get_device_status(torch.cuda.current_stream().cuda_stream) == FA_ERR_TIMEOUT
        elapsed = time.perf_counter() - t0
        assert elapsed < 2.0, f"the aborted launch took {elapsed:.2f} s"
        assert hooks.fa_get_device_status(None) == FA_OK   # read once, then cleared
        assert hooks.fa_test_set_withhold(-1) == FA_OK
        call.out.fill_(3.0)
        call.lse.fill_(5.0)
        g.replay()
        call.check()
        assert hooks.fa_get_device_status(None) == FA_OK
