"""The workspace of attention behind a prefix: what a call needs by its path and sizes, on the CPU."""
import pytest

import free_block_sparse_gb300 as fbs
from test_contexts_abi import PTR, pool, ref, t


@pytest.fixture(scope="module")
def lib():
    return fbs.lib()


def test_workspace_of_a_call(lib):
    most, of, own = (lib.sparge_cache4_prefix_attn_workspace_bytes, lib.sparge_cache4_prefix_attn_workspace_bytes_of,
                     lib.sparge_cache4_attn_workspace_bytes)
    few, many = (4, 32, 8, 1, 128), (64, 32, 8, 1, 128)
    # few sequences over a short prefix go alone, many over a long one share, a named path always does
    assert of(*few, 4096, fbs.SPARGE_PREFIX_AUTO) == own(*few) < 1 << 24 < most(*few)
    assert of(*many, 32768, fbs.SPARGE_PREFIX_AUTO) == most(*many) > own(*many)
    assert of(*few, 4096, fbs.SPARGE_PREFIX_SHARED) == most(*few)
    for path in (fbs.SPARGE_PREFIX_AUTO, fbs.SPARGE_PREFIX_SHARED):
        assert of(*many, 0, path) == own(*many)
        assert of(4, 32, 5, 1, 128, 4096, path) == 0 and of(*few, -16, path) == 0
    assert of(*few, 4096, 2) == 0


def test_calls_that_go_alone_take_the_smaller_one(lib):
    """The check of the workspace comes before that of the data, which is missing here: its error says which one failed."""
    import ctypes
    q = t(B=4, H=32, N=1, d=128)
    c = pool(n=64, page=64, H=8, d=128)
    arr = (ctypes.c_int32 * 64)()
    own = lib.sparge_cache4_attn_workspace_bytes(4, 32, 8, 1, 128)
    call = lambda n, path, ws: lib.sparge_cache4_prefix_attn(ref(q), ref(c), arr, n, None, 64, 64, None, 0.0, path, ref(q), PTR, ws, None)  # noqa: E731
    assert call(2, fbs.SPARGE_PREFIX_AUTO, own) == fbs.SPARGE_ERR_INVALID_ARG        # the table and lengths
    assert call(2, fbs.SPARGE_PREFIX_AUTO, own - 1) == fbs.SPARGE_ERR_WORKSPACE_TOO_SMALL
    assert call(2, fbs.SPARGE_PREFIX_SHARED, own) == fbs.SPARGE_ERR_WORKSPACE_TOO_SMALL
    assert call(0, fbs.SPARGE_PREFIX_SHARED, own) == fbs.SPARGE_ERR_INVALID_ARG
