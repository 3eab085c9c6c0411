"""The calls for long shared and multimodal contexts without a GPU: refusals (before anything is enqueued) and sizes."""
import ctypes
import math
import os

import pytest

import free_block_sparse_gb300 as fbs
from test_serving_abi import BAD, BIG, PTR, SMALL, UNSUP, pool, refused, t


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fbs.LIB_PATH):
        from free_block_sparse_gb300 import build
        build.build()
    return fbs.lib()


def ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), BAD), (dict(k=t(H=2, N=9)), BAD), (dict(q=t(dtype=3)), UNSUP), (dict(qo=t(H=5)), BAD), (dict(rot=24), BAD),
    (dict(rot=144), BAD), (dict(freq=None), BAD), (dict(eps=math.nan), BAD), (dict(n_axes=0), UNSUP), (dict(n_axes=5), UNSUP),
    (dict(axes=None), BAD), (dict(pos=None), BAD), (dict(sa=-1), BAD), (dict(sb=-8), BAD), (dict(ko=t(H=2, sn=136)), BAD),
])
def test_axes_refuses(lib, change, code):
    a = dict(q=t(), k=t(H=2), qo=t(ptr=2 * PTR), ko=t(H=2), rot=64, freq=PTR, eps=1e-6, pos=PTR, n_axes=3, sa=16, sb=8, axes=PTR)
    a.update(change)
    refused(lib, lib.sparge_qk_norm_rope_axes(ref(a["q"]), ref(a["k"]), a["pos"], a["n_axes"], a["sa"], a["sb"], a["axes"], a["freq"],
                                              a["rot"], 0, None, None, a["eps"], ref(a["qo"]), ref(a["ko"]), None), code)


@pytest.mark.parametrize("change,code", [
    (dict(c=None), BAD), (dict(c=pool(page=24)), UNSUP), (dict(c=pool(d=96)), UNSUP), (dict(bounds=None), BAD), (dict(bounds=PTR + 8), BAD),
    (dict(bytes=4 * 544 - 1), BAD), (dict(B=-1), UNSUP), (dict(B=65536), UNSUP), (dict(width=-1), BAD), (dict(stride=7), BAD),
    (dict(width=1 << 30, stride=1 << 30), BAD), (dict(table=None), BAD), (dict(lens=None), BAD), (dict(N=-1), BAD),
])
def test_bounds_update_refuses(lib, change, code):
    a = dict(c=pool(), table=PTR, B=2, width=8, stride=8, lens=PTR, N=3, bounds=PTR, bytes=4 * 544)
    a.update(change)
    refused(lib, lib.sparge_cache4_bounds_update(ref(a["c"]), a["table"], a["B"], a["width"], a["stride"], a["lens"], a["N"],
                                                 a["bounds"], a["bytes"], None), code)


@pytest.mark.parametrize("change,code", [
    (dict(c=None), BAD), (dict(bounds=None), BAD), (dict(bytes=100), BAD), (dict(n=-1), BAD), (dict(pages=None), BAD), (dict(hi=None), BAD),
    (dict(lo=PTR + 2), BAD), (dict(n=1 << 40), UNSUP),
])
def test_bounds_load_refuses(lib, change, code):
    a = dict(c=pool(), bounds=PTR, bytes=4 * 544, pages=PTR, n=5, hi=PTR, lo=PTR)
    a.update(change)
    refused(lib, lib.sparge_cache4_bounds_load(ref(a["c"]), a["bounds"], a["bytes"], a["pages"], a["n"], a["hi"], a["lo"], None), code)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), BAD), (dict(q=t(H=3)), UNSUP), (dict(q=t(d=64)), BAD), (dict(q=t(H=130)), UNSUP), (dict(c=pool(page=24)), UNSUP),
    (dict(bounds=None), BAD), (dict(bytes=99), BAD), (dict(width=-1), BAD), (dict(stride=7), BAD), (dict(width=32769, stride=32769), UNSUP),
    (dict(table=None), BAD), (dict(lens=None), BAD), (dict(keep=-1), BAD), (dict(keep=1 << 30), BAD), (dict(first=-1), BAD),
    (dict(last=0), BAD), (dict(keep=3, first=2, last=2), BAD), (dict(first=1 << 62, last=1 << 62), BAD), (dict(pages=None), BAD),
    (dict(out=None), BAD), (dict(out=3 * PTR), BAD), (dict(ws=None), SMALL), (dict(wsb=2 * 8 * 2 * 8 * 4 - 1), SMALL), (dict(ws=PTR + 16), BAD),
])
def test_select_refuses(lib, change, code):
    a = dict(q=t(), c=pool(), bounds=PTR, bytes=4 * 544, table=PTR, width=8, stride=8, lens=3 * PTR, keep=6, first=1, last=1, pages=PTR,
             out=2 * PTR, ws=PTR, wsb=BIG)
    a.update(change)
    refused(lib, lib.sparge_cache4_select(ref(a["q"]), ref(a["c"]), a["bounds"], a["bytes"], a["table"], a["width"], a["stride"],
                                          a["lens"], a["keep"], a["first"], a["last"], a["pages"], a["out"], a["ws"], a["wsb"], None), code)


@pytest.mark.parametrize("change,code", [
    (dict(q=t(H=3), o=t(H=3)), UNSUP), (dict(q=t(d=64), o=t(d=64)), BAD), (dict(o=t(N=9)), BAD), (dict(c=pool(page=24)), UNSUP),
    (dict(keep=-1), BAD), (dict(keep=1 << 30), BAD), (dict(scale=-1.0), BAD), (dict(scale=math.nan), BAD), (dict(pages=None), BAD),
    (dict(lens=None), BAD), (dict(ws=None), SMALL), (dict(wsb=100), SMALL), (dict(ws=PTR + 16), BAD), (dict(q=None), BAD),
])
def test_pages_attn_refuses(lib, change, code):
    a = dict(q=t(), o=t(), c=pool(), pages=PTR, keep=8, lens=PTR, scale=0.0, ws=PTR, wsb=BIG)
    a.update(change)
    refused(lib, lib.sparge_cache4_pages_attn(ref(a["q"]), ref(a["c"]), a["pages"], a["keep"], a["lens"], a["scale"], ref(a["o"]),
                                              a["ws"], a["wsb"], None), code)


@pytest.mark.parametrize("change,code", [
    (dict(q=t(H=3), o=t(H=3)), UNSUP), (dict(q=t(d=64), o=t(d=64)), BAD), (dict(o=t(N=9)), BAD), (dict(c=pool(page=24)), UNSUP),
    (dict(n=-1), BAD), (dict(n=9), BAD), (dict(prefix=None), BAD), (dict(width=-1), BAD), (dict(stride=7), BAD),
    (dict(width=1 << 30, stride=1 << 30), BAD), (dict(scale=-1.0), BAD), (dict(scale=math.inf), BAD), (dict(table=None), BAD),
    (dict(lens=None), BAD), (dict(ws=None), SMALL), (dict(wsb=100), SMALL), (dict(ws=PTR + 16), BAD), (dict(q=None), BAD),
    (dict(path=-1), BAD), (dict(path=2), BAD),
])
def test_prefix_attn_refuses(lib, change, code):
    a = dict(q=t(), o=t(), c=pool(), prefix=PTR, n=3, table=PTR, width=8, stride=8, lens=PTR, scale=0.0, ws=PTR, wsb=BIG, path=0)
    a.update(change)
    refused(lib, lib.sparge_cache4_prefix_attn(ref(a["q"]), ref(a["c"]), a["prefix"], a["n"], a["table"], a["width"], a["stride"],
                                               a["lens"], a["scale"], a["path"], ref(a["o"]), a["ws"], a["wsb"], None), code)


def test_calls_of_nothing(lib):
    """Empty batches and empty queries need no data."""
    e, c = t(ptr=None, N=0), pool(ptr=None, n=0)
    assert lib.sparge_qk_norm_rope_axes(ref(e), ref(e), None, 1, 0, 0, None, PTR, 64, 0, None, None, 1e-6, ref(e), ref(e), None) == 0
    assert lib.sparge_cache4_bounds_update(ref(c), None, 0, 0, 0, None, 1, None, 0, None) == 0
    assert lib.sparge_cache4_bounds_load(ref(c), None, 0, None, 0, None, None, None) == 0
    assert lib.sparge_cache4_select(ref(e), ref(c), None, 0, None, 0, 0, PTR, 2, 1, 1, None, None, None, 0, None) == 0
    assert lib.sparge_cache4_pages_attn(ref(e), ref(c), None, 4, None, 0.0, ref(e), PTR, BIG, None) == 0
    assert lib.sparge_cache4_prefix_attn(ref(e), ref(c), None, 0, None, 0, 0, None, 0.0, 0, ref(e), PTR, BIG, None) == 0


def test_sizes(lib):
    for H, d, row in ((8, 128, 2080), (1, 64, 160), (3, 64, 416), (5, 128, 1312)):
        assert lib.sparge_cache4_bounds_bytes(1, H, d) == row and lib.sparge_cache4_bounds_bytes(1 << 24, H, d) == row << 24
    for bad in ((-1, 2, 128), (1, 0, 128), (1, 2, 96), (1, 65536, 64)):
        assert lib.sparge_cache4_bounds_bytes(*bad) == 0
    assert lib.sparge_cache4_select_workspace_bytes(3, 8, 2, 1001) == 3 * 8 * 2 * 1004 * 4
    for bad in ((-1, 8, 2, 10), (3, 0, 2, 10), (3, 8, -1, 10), (3, 8, 2, 32769), (65535, 65535, 1, 10)):
        assert lib.sparge_cache4_select_workspace_bytes(*bad) == 0
    for f in (lib.sparge_cache4_pages_attn_workspace_bytes, lib.sparge_cache4_prefix_attn_workspace_bytes):
        assert f(4, 32, 8, 1, 128) > 0 and f(4, 32, 5, 1, 128) == 0 and f(4, 32, 8, 1, 96) == 0 and f(-1, 32, 8, 1, 128) == 0
        assert f(65536, 32, 8, 1, 128) == 0 and f(65535, 32, 32, 1 << 30, 128) == 0


def test_rope_axes():
    pytest.importorskip("torch")
    assert fbs.rope_axes((2, 0, 3), device="cpu").tolist() == [0, 0, 2, 2, 2]
    assert fbs.rope_axes((2, 0, 3), woven=True, device="cpu").tolist() == [0, 2, 0, 2, 2]
    assert fbs.rope_axes((), woven=True, device="cpu").numel() == 0
    for woven in (False, True):
        with pytest.raises(ValueError):
            fbs.rope_axes((3, -1), woven=woven, device="cpu")


def test_grid_positions_on_the_host():
    pytest.importorskip("torch")
    pos = fbs.rope_grid_positions(2, 1, 2, 2, device="cpu")
    assert pos.tolist() == [[[0, 1, 2, 2, 2, 2]], [[0, 1, 2, 2, 3, 3]], [[0, 1, 2, 3, 2, 3]]]


def test_binding_refuses_host_tensors(lib):
    torch = pytest.importorskip("torch")
    t4 = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fbs.qk_norm_rope_axes(t4, t4, i, i, i), lambda: fbs.cache4_bounds_update(t4, i, i, 1, i),
                 lambda: fbs.cache4_bounds_load(t4, i, i), lambda: fbs.cache4_select(t4, t4, i, i, i, 1),
                 lambda: fbs.cache4_pages_attn(t4, t4, i, i), lambda: fbs.cache4_prefix_attn(t4, t4, i, i, i)):
        with pytest.raises(ValueError):
            call()
    for bad in ((-1, 2, 128), (1, 0, 128), (1, 2, 96)):
        with pytest.raises(ValueError):
            fbs.cache4_bounds(*bad, device="cpu")
    assert fbs.cache4_bounds(3, 8, 128, device="cpu").shape == (3, 2080)
    assert fbs.rope_axes((2, 0, 3), device="cpu").tolist() == [0, 0, 2, 2, 2]
    assert fbs.rope_axes((2, 0, 3), woven=True, device="cpu").tolist() == [0, 2, 0, 2, 2]
