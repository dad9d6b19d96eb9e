"""Host-side refusals of fa_fwd_paged at its limits (no kernel is launched)."""
import pytest

from exact_attention_113_b200.build import build
import exact_attention_113_b200 as fa
from tests.test_paged_host import _paged


@pytest.fixture(scope="module")
def lib():
    build()
    return fa.load()


def test_batches_too_large_to_walk_are_refused(lib):
    assert _paged(B=(1 << 24) + 1, H_kv=1) == -2
    assert _paged(B=1 << 24, H_kv=1, T=0) == 0
