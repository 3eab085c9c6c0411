"""The serving calls without a GPU: refusals (before anything is enqueued), sizes and struct layout."""
import ctypes
import math
import os

import pytest

import free_block_sparse_gb300 as fbs

BAD, UNSUP, SMALL = fbs.SPARGE_ERR_INVALID_ARG, fbs.SPARGE_ERR_UNSUPPORTED, fbs.SPARGE_ERR_WORKSPACE_TOO_SMALL
PTR = 0x10000
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fbs.LIB_PATH):
        from free_block_sparse_gb300 import build
        build.build()
    return fbs.lib()


def t(ptr=PTR, B=2, H=4, N=8, d=128, dtype=fbs.SPARGE_BF16, sn=None):
    sn = d if sn is None else sn
    rows = max(N, 1) * sn
    return fbs.sparge_tensor(ptr, dtype, 0, B, H, N, d, H * rows, rows, sn)


def pool(ptr=PTR, n=4, page=64, H=2, d=128):
    return fbs.sparge_cache4(ptr, n, page, H, d, 0)


def refused(lib, rc, code):
    assert rc == code, (rc, lib.sparge_last_error())
    assert lib.sparge_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(q=None), BAD), (dict(k=t(H=2, N=9)), BAD), (dict(k=t(H=2, d=64)), BAD), (dict(q=t(dtype=3)), UNSUP),
    (dict(q=t(d=96), k=t(d=96)), UNSUP), (dict(qo=t(H=5)), BAD), (dict(ko=t(H=2, sn=136)), BAD), (dict(rot=24), BAD),
    (dict(rot=144), BAD), (dict(rot=-16), BAD), (dict(freq=None), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD),
    (dict(eps=math.inf), BAD), (dict(q=t(ptr=PTR + 2)), BAD), (dict(qo=None), BAD),
])
def test_norm_rope_refuses(lib, change, code):
    a = dict(q=t(), k=t(H=2), qo=t(ptr=2 * PTR), ko=t(H=2), rot=64, freq=PTR, eps=1e-6)
    a.update(change)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    refused(lib, lib.sparge_qk_norm_rope(ref(a["q"]), ref(a["k"]), None, 0, a["freq"], a["rot"], 0, None, None, a["eps"],
                                         ref(a["qo"]), ref(a["ko"]), None), code)


def test_norm_rope_of_nothing(lib):
    e = t(ptr=None, N=0)
    assert lib.sparge_qk_norm_rope(*(ctypes.byref(e),) * 2, None, 0, PTR, 64, 0, None, None, 1e-6, ctypes.byref(e),
                                   ctypes.byref(e), None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(lens=None), BAD), (dict(new=None), BAD), (dict(R=-1), BAD), (dict(N=-1), BAD), (dict(page=48), UNSUP),
    (dict(page=8), UNSUP), (dict(page=512), UNSUP), (dict(R=65536), UNSUP), (dict(N=1 << 31), UNSUP),
    (dict(stride=7), BAD), (dict(table=None), BAD), (dict(free=None), BAD), (dict(n_free=-1), BAD), (dict(width=-1), BAD),
])
def test_cache_tables_refuses(lib, change, code):
    a = dict(lens=PTR, new=PTR, R=3, N=2, page=64, free=PTR, n_free=5, table=PTR, width=8, stride=8)
    a.update(change)
    refused(lib, lib.sparge_cache_tables(a["lens"], a["new"], a["R"], a["N"], a["page"], a["free"], a["n_free"], a["table"],
                                         a["width"], a["stride"], PTR, PTR, PTR, PTR, None), code)


@pytest.mark.parametrize("lens,new,kv", [(PTR, 2 * PTR, PTR), (2 * PTR, PTR, PTR)])
def test_cache_tables_refuses_lengths_in_place(lib, lens, new, kv):
    """Every CTA reads the lengths of the requests in front of its own: none may be overwritten meanwhile."""
    refused(lib, lib.sparge_cache_tables(lens, new, 3, 2, 64, 4 * PTR, 5, 5 * PTR, 8, 8, 6 * PTR, 7 * PTR, kv, 8 * PTR, None), BAD)
    assert b"kv_lens" in lib.sparge_last_error()


@pytest.mark.parametrize("load", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(c=None), BAD), (dict(c=pool(H=3)), BAD), (dict(c=pool(d=64)), BAD), (dict(c=pool(d=96)), UNSUP),
    (dict(c=pool(page=8)), UNSUP), (dict(c=pool(page=80)), UNSUP), (dict(c=pool(n=-1)), BAD), (dict(c=pool(n=1 << 40)), UNSUP),
    (dict(c=pool(ptr=None)), BAD), (dict(c=pool(ptr=PTR + 8)), BAD), (dict(v=t(H=2, N=9)), BAD), (dict(k=None), BAD),
    (dict(slots=None), BAD), (dict(c=pool(H=0)), BAD),
])
def test_store_and_load_refuse(lib, load, change, code):
    a = dict(k=t(H=2), v=t(H=2), slots=PTR, c=pool())
    a.update(change)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    k, v, c = ref(a["k"]), ref(a["v"]), ref(a["c"])
    rc = lib.sparge_cache4_load(c, a["slots"], 0, k, v, None) if load else lib.sparge_cache4_store(k, v, a["slots"], c, None)
    refused(lib, rc, code)


@pytest.mark.parametrize("change,code", [
    (dict(q=t(H=3), o=t(H=3)), UNSUP), (dict(q=t(d=64), o=t(d=64)), BAD), (dict(o=t(N=9)), BAD), (dict(c=pool(page=24)), UNSUP),
    (dict(window=-1), BAD), (dict(window=0, sinks=3), BAD), (dict(sinks=-1, window=5), BAD), (dict(window=1 << 31), BAD),
    (dict(scale=-1.0), BAD), (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(width=-1), BAD),
    (dict(width=9), BAD), (dict(width=1 << 30, stride=1 << 30), BAD), (dict(ws=None), SMALL), (dict(wsb=100), SMALL),
    (dict(ws=PTR + 16), BAD), (dict(table=None), BAD), (dict(lens=None), BAD), (dict(q=None), BAD),
])
def test_cache_attn_refuses(lib, change, code):
    a = dict(q=t(), o=t(), c=pool(), table=PTR, width=8, stride=8, lens=PTR, window=0, sinks=0, scale=0.0, ws=PTR, wsb=BIG)
    a.update(change)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    refused(lib, lib.sparge_cache4_attn(ref(a["q"]), ref(a["c"]), a["table"], a["width"], a["stride"], a["lens"], a["window"],
                                        a["sinks"], a["scale"], ref(a["o"]), a["ws"], a["wsb"], None), code)


@pytest.mark.parametrize("change,code", [
    (dict(window=0), BAD), (dict(window=-5), BAD), (dict(sinks=-1), BAD), (dict(q=t(N=17)), BAD), (dict(v=t(H=2, N=15)), BAD),
    (dict(o=t(H=2)), BAD), (dict(q=t(H=3), o=t(H=3)), UNSUP), (dict(scale=math.nan), BAD), (dict(scale=-0.5), BAD),
    (dict(ws=None), SMALL), (dict(wsb=64), SMALL), (dict(ws=PTR + 128), BAD), (dict(k=None), BAD), (dict(q=t(dtype=2)), UNSUP),
])
def test_window_attn_refuses(lib, change, code):
    a = dict(q=t(), k=t(H=2, N=16), v=t(H=2, N=16), o=t(), window=4, sinks=1, scale=0.0, ws=PTR, wsb=BIG)
    a.update(change)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    refused(lib, lib.sparge_window_attn(ref(a["q"]), ref(a["k"]), ref(a["v"]), a["window"], a["sinks"], a["scale"], ref(a["o"]),
                                        a["ws"], a["wsb"], None), code)


def test_sizes(lib):
    for d in (64, 128):
        for page in (16, 32, 64, 128, 256):
            assert lib.sparge_cache4_bytes(3, page, 2, d) == 3 * 2 * page * (d + d // 8)
    assert lib.sparge_cache4_bytes(1 << 20, 256, 8, 128) == (1 << 20) * 256 * 8 * 144      # past 32 bits
    for bad in ((-1, 64, 2, 128), (3, 8, 2, 128), (3, 48, 2, 128), (3, 64, 0, 128), (3, 64, 2, 96)):
        assert lib.sparge_cache4_bytes(*bad) == 0
    # partial rows of every CTA and item
    assert lib.sparge_cache4_attn_workspace_bytes(4, 32, 8, 1, 128) >= (608 + 32) * 8 * 130 * 4
    assert lib.sparge_cache4_attn_workspace_bytes(4, 32, 5, 1, 128) == 0
    assert lib.sparge_cache4_attn_workspace_bytes(4, 32, 8, 1, 96) == 0
    assert fbs.workspace_bytes(fbs.SPARGE_OP_WINDOW_ATTN, 1, 32, 8, 32768, 128) >= 2 * 8 * 32768 * 128
    assert fbs.workspace_bytes(fbs.SPARGE_OP_WINDOW_ATTN, 1, 32, 8, 32768, 96) == 0


def test_window_workspace_holds_v_and_the_decoding_rows(lib):
    for B, Hkv, Nk, d in ((1, 1, 100, 64), (1, 2, 131072, 128), (3, 4, 5000, 64), (16, 8, 32768, 128)):
        have = fbs.workspace_bytes(fbs.SPARGE_OP_WINDOW_ATTN, B, Hkv, Hkv, Nk, d)
        slots = B * Hkv * 8 + 304          # row tiles of 128 rows, and the CTAs
        assert have >= 2 * B * Hkv * Nk * d and have >= slots * 16 * (d + 2) * 4


def test_cache4_struct_layout(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"sparge.h\"\nint main(void) {\n"
                   "  printf(\"%zu %zu %zu %zu %zu\\n\", sizeof(sparge_cache4), offsetof(sparge_cache4, n_pages),\n"
                   "         offsetof(sparge_cache4, page_size), offsetof(sparge_cache4, H), offsetof(sparge_cache4, d));\n"
                   "  return 0;\n}\n")
    exe = tmp_path / "layout"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    C = fbs.sparge_cache4
    assert got == [ctypes.sizeof(C), C.n_pages.offset, C.page_size.offset, C.H.offset, C.d.offset]


def test_binding_refuses_host_tensors(lib):
    """The Python calls take CUDA tensors alone and say so, without a GPU as well."""
    torch = pytest.importorskip("torch")
    t4 = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fbs.window_attn(t4, t4, t4, 1), lambda: fbs.qk_norm_rope(t4, t4), lambda: fbs.cache4_store(t4, t4, i, i),
                 lambda: fbs.cache4_load(t4, i), lambda: fbs.cache4_attn(t4, t4, i, i), lambda: fbs.cache_tables(i, i, i, i, 16, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fbs.window_attn(1, t4, t4, 1)
    with pytest.raises(TypeError):
        fbs._load_binding().cache4_store(t4)
