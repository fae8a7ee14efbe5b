"""Host-side checks of the storing calls given no tokens: an empty tensor's pointer is NULL, but
values without a plane are refused as with tokens."""
import ctypes

import pytest

import sparse_attention_indexer_packed_gb300 as idx
from test_ops_abi_cpu import FAKE, pool

by = ctypes.byref


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return idx.lib()


def calls(L, k, v, with_plane):
    """Status of the three calls with 0 tokens: bf16, e4m3 and NVFP4 planes."""
    for dtype in (0, 1, 2):
        p = pool(dtype)
        vp = by(p) if with_plane else None
        if dtype == 2:
            yield L.idx_store_kv_nvfp4(k, v, 256, 256, None, 0, 2, by(p), vp, 1.0, 1.0, None)
        else:
            yield L.idx_store_kv(k, v, 256, 256, None, 0, 2, by(p), vp, None)
        yield L.idx_norm_rope_store(None, 0, 0, k, 256, v, 256, 2, None, None, 0.0, None, None, 0, None, None,
                                    by(p), vp, 1.0, 1.0, None)


@pytest.mark.parametrize("k,v,with_plane", [(None, None, True), (None, None, False), (FAKE, FAKE, True)])
def test_no_tokens_is_a_no_op(L, k, v, with_plane):
    assert set(calls(L, k, v, with_plane)) == {0}


@pytest.mark.parametrize("k", [None, FAKE])
def test_values_without_a_plane_are_refused(L, k):
    assert set(calls(L, k, FAKE, False)) == {-1}
    assert b"together" in L.idx_last_error()
