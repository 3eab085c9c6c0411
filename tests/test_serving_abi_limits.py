"""The serving calls at the ends of their sizes, without a GPU: empty calls and sizes past what a call takes."""
import ctypes
import os

import pytest

import free_block_sparse_gb300 as fbs


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fbs.LIB_PATH):
        from free_block_sparse_gb300 import build
        build.build()
    return fbs.lib()


def t(B, H, N, d, strides, ptr=None):
    return ctypes.byref(fbs.sparge_tensor(ptr, fbs.SPARGE_BF16, 0, B, H, N, d, *strides))


def test_norm_rope_of_nothing_takes_any_strides(lib):
    """Tensors without tokens have no data, so two of them at the same (null) address are not one in place."""
    q, k = t(2, 4, 0, 64, (256, 64, 256)), t(2, 2, 0, 64, (128, 64, 128))
    a, b = t(2, 4, 0, 64, (256, 64, 64)), t(2, 2, 0, 64, (128, 64, 64))
    assert lib.sparge_qk_norm_rope(q, k, None, 0, None, 0, 0, None, None, 1e-6, a, b, None) == 0, lib.sparge_last_error()
