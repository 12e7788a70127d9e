"""Which rows the expert layer takes: the workspace query and the two calls agree, and the documented ranges hold."""
import pytest

from bit_quantized_gemv_tq1_gb300 import _lib as L
from bit_quantized_gemv_tq1_gb300 import build as B
from tests.test_step_host import UNSUPPORTED, WORKSPACE, moe

BATCHES = [(1, 1, 1), (2, 2, 2), (8, 2, 7), (128, 8, 512), (1024, 32, 128), (1024, 1, 4096)]  # experts, top_k, tokens


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.library()


def refused(lib, fn, n, k, f, t, top_k):
    """Whether the call does not take such rows; the workspace is too small, so that nothing is launched."""
    code = moe(lib, fn, n=n, k=k, f=f, t=t, top_k=top_k, ws_bytes=0)
    assert code in (UNSUPPORTED, WORKSPACE)
    return code == UNSUPPORTED


@pytest.mark.parametrize("n,top_k,t", BATCHES)
def test_the_query_is_zero_where_both_calls_refuse(lib, n, top_k, t):
    seen = set()
    for k in list(range(256, 65537, 1280)) + [10240, 10752, 11008, 12800, 13056, 14336, 16384, 16640, 19456, 22016, 22528, 65536]:
        for f in (256, 4096, 10240, 49152, 55040, 58624, 65536):
            both = [refused(lib, fn, n, k, f, t, top_k) for fn in ("tq1_moe", "tq2_moe")]
            assert (L.tq1_moe_workspace_size(n, k, f, t, top_k) == 0) == all(both)
            assert both[1] or not both[0]  # what TQ2_0 takes, TQ1_0 does
            seen.add(tuple(both))
    assert seen == {(False, False), (False, True), (True, True)}


@pytest.mark.parametrize("fn", ["tq1_moe", "tq2_moe"])
@pytest.mark.parametrize("n,top_k,t", BATCHES)
def test_documented_rows_are_taken(lib, fn, n, top_k, t):
    for k, f in ((16384, 49152), (16384, 256), (256, 49152), (10240, 65536), (256, 65536), (10496, 49152)):
        assert not refused(lib, fn, n, k, f, t, top_k)


def test_the_query_does_not_shrink_with_the_batch(lib):
    for k, f in ((10240, 65536), (16384, 49152), (512, 256)):
        sizes = [L.tq1_moe_workspace_size(64, k, f, t, 2) for t in (0, 1, 2, 9, 100, 2048)]
        assert sizes == sorted(sizes)
