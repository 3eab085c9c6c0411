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


@pytest.mark.parametrize("shape", [(65535, 65535, 65535, 1 << 30, 128), (1, 65535, 1, 1 << 30, 64), (65535, 65535, 65535, 1, 64),
                                   (4096, 32, 32, 1 << 30, 128)])
def test_workspace_of_a_cache_attention_that_is_too_large(lib, shape):
    """Sizes that the call refuses have no workspace (they do not wrap around to a small one)."""
    assert lib.sparge_cache4_attn_workspace_bytes(*shape) == 0
    B, Hq, Hkv, Nq, d = shape
    row = Hq * d
    q = t(B, Hq, Nq, d, (Nq * row, d, row), ptr=1 << 16)
    pool = fbs.sparge_cache4(1 << 16, 4, 16, Hkv, d, 0)
    rc = lib.sparge_cache4_attn(q, ctypes.byref(pool), 1 << 16, 4, 4, 1 << 16, 0, 0, 0.0, q, 1 << 16, (1 << 64) - 1, None)
    assert rc == fbs.SPARGE_ERR_UNSUPPORTED, (rc, lib.sparge_last_error())


def test_workspace_of_the_largest_cache_attentions(lib):
    """What the call takes has a workspace of at least its partial rows."""
    for B, Hq, Hkv, Nq, d in ((65535, 256, 128, 8, 128), (1, 1, 1, 1 << 30, 64), (256, 64, 8, 1, 128)):
        rows = Hq // Hkv * Nq
        assert lib.sparge_cache4_attn_workspace_bytes(B, Hq, Hkv, Nq, d) >= B * Hkv * rows * (d + 2) * 4
