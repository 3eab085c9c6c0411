"""GB300 (sm_103a) SpargeAttn: two-stage sparse attention forward behind a C ABI.

Thin Python binding over ``libsparge.so`` (see include/sparge.h for the contract of every
call).  This module only marshals arguments: torch provides device memory and the current CUDA
stream, every step of the computation runs in the library's CUDA kernels.  There is no CPU
path: if the library is missing or no CUDA device is present the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsparge.so")

SPARGE_OK = 0
SPARGE_ERR_INVALID_ARG = -1
SPARGE_ERR_UNSUPPORTED = -2
SPARGE_ERR_WORKSPACE_TOO_SMALL = -3
SPARGE_ERR_CUDA = -4
SPARGE_ERR_DEVICE_TIMEOUT = -5
SPARGE_BF16 = 1
SPARGE_PREFIX_AUTO = 0
SPARGE_PREFIX_SHARED = 1
SPARGE_PRECISION_BF16 = 0
SPARGE_PRECISION_Q8 = 1
SPARGE_PRECISION_Q8_FP8PV = 2
SPARGE_PRECISION_BF16_FP8PV = 3
# precisions with an 8-bit product: d = 128 and the 8-bit workspace (SPARGE_OP_*_Q8)
PRECISIONS_8BIT = (SPARGE_PRECISION_Q8, SPARGE_PRECISION_Q8_FP8PV, SPARGE_PRECISION_BF16_FP8PV)
SPARGE_OP_PREDICT_MASK = 1
SPARGE_OP_BLOCK_SPARSE_ATTN = 2
SPARGE_OP_ATTN = 3
SPARGE_OP_BLOCK_SPARSE_ATTN_Q8 = 4
SPARGE_OP_ATTN_Q8 = 5
SPARGE_OP_WINDOW_ATTN = 6
SPARGE_OP_TOKEN_ORDER = 0x100  # flag OR-ed into an op: room for token-ordered copies of Q and K
SPARGE_TOPK_CUMULATIVE = 0      # topk is a cumulative probability fraction (default)
SPARGE_TOPK_COUNT = 1           # topk is a fraction of the valid blocks to keep
SPARGE_TOPK_HYBRID = 2          # the count set of topk united with the cumulative set of topp
QBLK, KBLK = 128, 64


class SpargeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("sparge error %d: %s" % (code, msg))
        self.code = code


class sparge_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("pad_", ctypes.c_int32),
                ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64), ("d", ctypes.c_int64),
                ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64), ("stride_n", ctypes.c_int64)]


class sparge_params(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_float), ("lambda_", ctypes.c_float), ("scale", ctypes.c_float),
                ("precision", ctypes.c_int32), ("stats", ctypes.c_void_p), ("timing_events", ctypes.c_void_p),
                ("topk_per_head", ctypes.c_void_p), ("theta_per_head", ctypes.c_void_p),
                ("lambda_per_head", ctypes.c_void_p), ("token_order", ctypes.c_void_p), ("topk_mode", ctypes.c_int32),
                ("topp", ctypes.c_float)]


class sparge_cache4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("H", ctypes.c_int32), ("d", ctypes.c_int32), ("pad_", ctypes.c_int32)]


_lib = None

EXPORTS = {
    "sparge_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] + [ctypes.c_int64] * 5),
    "sparge_predict_mask": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_float,
                                           ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.c_void_p]),
    "sparge_predict_mask_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_int,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                              ctypes.c_void_p]),
    "sparge_block_sparse_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_block_sparse_attn_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                   ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                   ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_int,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_attn_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_int,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_permute_tokens": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_unpermute_tokens": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_hilbert_perm_2d": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "sparge_hilbert_perm_3d": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "sparge_predict_mask_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_float,
                                                   ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_window_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_qk_norm_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p]),
    "sparge_cache4_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "sparge_cache_tables": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_cache4_store": (ctypes.c_int, [ctypes.c_void_p] * 5),
    "sparge_cache4_load": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_cache4_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64] * 5),
    "sparge_cache4_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                          ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p]),
    "sparge_qk_norm_rope_axes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                                ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_cache4_bounds_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int]),
    "sparge_cache4_bounds_update": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                                   ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                                   ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_cache4_bounds_load": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                                 ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "sparge_cache4_select": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_cache4_select_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64] * 4),
    "sparge_cache4_pages_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64] * 5),
    "sparge_cache4_pages_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                                ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_cache4_prefix_attn_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64] * 5),
    "sparge_cache4_prefix_attn_workspace_bytes_of": (ctypes.c_size_t, [ctypes.c_int64] * 6 + [ctypes.c_int]),
    "sparge_cache4_prefix_attn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                                 ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                                 ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_size_t, ctypes.c_void_p]),
    "sparge_selftest_bounded_wait": (ctypes.c_int, [ctypes.c_int64, ctypes.c_void_p]),
    "sparge_last_error": (ctypes.c_char_p, []),
    "sparge_get_device_status": (ctypes.c_int, [ctypes.c_void_p]),
}


def lib():
    """Load libsparge.so (built by ``free_block_sparse_gb300.build``); raise if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libsparge.so is not built (%s); run free_block_sparse_gb300.build.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(rc: int):
    if rc != SPARGE_OK:
        raise SpargeError(rc, lib().sparge_last_error().decode())


_torch_module = None


def _torch():
    """torch, imported on first use (an import statement in every call costs about half a microsecond)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream():
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


_binding_module = None


def _load_binding():
    """The compiled binding of the serving calls (csrc/binding.cpp).  They are made once per token and layer, and at
    decoding sizes a call through ctypes takes the host longer than its kernels take the GPU."""
    global _binding_module
    if _binding_module is None:
        lib()     # the library the binding calls into
        _torch()  # and torch's own libraries
        if not os.path.exists(os.path.join(_PKG, "_binding.so")):
            raise RuntimeError("_binding.so is not built (it needs torch at build time); run free_block_sparse_gb300.build.build()")
        from . import _binding as m
        m.set_error(SpargeError)
        _binding_module = m
    return _binding_module


def _desc(t) -> sparge_tensor:
    torch = _torch()
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError("expected a CUDA tensor")
    if t.dtype != torch.bfloat16 or t.dim() != 4 or t.stride(-1) != 1:
        raise TypeError("expected a bf16 (B, H, N, d) tensor with contiguous last dim")
    B, H, N, d = t.shape
    sb, sh, sn, _ = t.stride()
    return sparge_tensor(t.data_ptr(), SPARGE_BF16, 0, B, H, N, d, sb, sh, sn)


def workspace_bytes(op: int, B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(lib().sparge_workspace_bytes(op, B, Hq, Hkv, N, d))


def n_blocks(N: int):
    return -(-N // QBLK), -(-N // KBLK)


def _workspace(op, q, k, ws):
    torch = _torch()
    B, Hq, Nq, d = q.shape
    need = workspace_bytes(op, B, Hq, k.shape[1], max(Nq, k.shape[2]), d)   # N: an upper bound of both
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    return ws


def predict_mask(q, k, topk: float, theta: float = 0.5, causal: bool = False, ws=None, mask=None):
    """Stage 1: the (B, Hq, ceil(Nq/128), ceil(Nk/64)) uint8 block mask."""
    torch = _torch()
    B, Hq, Nq, d = q.shape
    nqb, nkb = -(-Nq // 128), -(-k.shape[2] // 64)
    if mask is None:
        mask = torch.empty((B, Hq, nqb, nkb), dtype=torch.uint8, device=q.device)
    ws = _workspace(SPARGE_OP_PREDICT_MASK, q, k, ws)
    dq, dk = _desc(q), _desc(k)
    _check(lib().sparge_predict_mask(ctypes.byref(dq), ctypes.byref(dk), float(topk), float(theta), int(causal),
                                     mask.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return mask


def predict_mask_ex(q, k, topk: float, causal: bool = False, theta: float = 0.5, scale: float = 0.0,
                    topk_per_head=None, theta_per_head=None, ws=None, mask=None, events=None, token_order=None,
                    topk_mode: int = SPARGE_TOPK_CUMULATIVE, topp: float = 1.0):
    """predict_mask with an explicit pooled-score scale, optional per-query-head topk and theta
    (float32 CUDA tensors of Hq entries), optional timing events ([0]-[3] are recorded), an
    optional token order (int32 CUDA tensor of N entries; the mask refers to the reordered
    sequence) and the reading of topk (topk_mode; topp is the top-p mass of the hybrid rule)."""
    torch = _torch()
    B, Hq, Nq, _ = q.shape
    if mask is None:
        mask = torch.empty((B, Hq, -(-Nq // 128), -(-k.shape[2] // 64)), dtype=torch.uint8, device=q.device)
    ws = _workspace(SPARGE_OP_PREDICT_MASK | (SPARGE_OP_TOKEN_ORDER if token_order is not None else 0), q, k, ws)
    p = _params(theta, -math.inf, scale, SPARGE_PRECISION_BF16, None, events, topk_per_head, theta_per_head,
                order=token_order, topk_mode=topk_mode, topp=topp)
    dq, dk = _desc(q), _desc(k)
    _check(lib().sparge_predict_mask_ex(ctypes.byref(dq), ctypes.byref(dk), float(topk), int(causal), ctypes.byref(p),
                                        mask.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return mask


def predict_ws_views(ws, B, Hq, Hkv, N, d, Nk=None):
    """Views of the stage-1 workspace after predict_mask: muQ (B,Hq,nqb,d), sQ (B,Hq,nqb),
    muK (B,Hkv,nkb,d), sK (B,Hkv,nkb) and the scaled pooled scores S (B,Hq,nqb,nkb), following
    the layout the library writes (regions 256-byte aligned; fp32 except the bf16 hi/lo copies of
    the means, which are skipped here).  N is the query length, Nk the key length (default N)."""
    torch = _torch()
    nqb = n_blocks(N)[0]
    nkb = n_blocks(N if Nk is None else Nk)[1]
    nkb_pad = -(-nkb // 4) * 4
    u8 = ws if ws.dtype == torch.uint8 else ws.view(torch.uint8)

    def take(off, nbytes):
        return u8[off:off + nbytes], off + ((nbytes + 255) // 256) * 256

    off = 0
    muQ, off = take(off, 4 * B * Hq * nqb * d)
    sQ, off = take(off, 4 * B * Hq * nqb)
    muK, off = take(off, 4 * B * Hkv * nkb * d)
    sK, off = take(off, 4 * B * Hkv * nkb_pad)
    _, off = take(off, 2 * B * Hq * nqb * d)
    _, off = take(off, 2 * B * Hq * nqb * d)
    _, off = take(off, 2 * B * Hkv * nkb * d)
    _, off = take(off, 2 * B * Hkv * nkb * d)
    S, off = take(off, 4 * B * Hq * nqb * nkb_pad)
    f = lambda t: t.view(torch.float32)
    return (f(muQ).view(B, Hq, nqb, d), f(sQ).view(B, Hq, nqb), f(muK).view(B, Hkv, nkb, d),
            f(sK).view(B, Hkv, nkb_pad)[..., :nkb], f(S).view(B, Hq, nqb, nkb_pad)[..., :nkb])


def q8_ws_views(ws, B, Hq, Hkv, N, d):
    """Views of the 8-bit attention workspace after block_sparse_attn with an 8-bit precision: q8
    (B,Hq,N,d) and k8 (B,Hkv,N,d) e4m3 codes (uint8), v8 (B,Hkv,d,npad) channel-major e4m3 codes
    (meaningful after SPARGE_PRECISION_Q8_FP8PV), sq (B,Hq,nqb), sk (B,Hkv,nkb), kmean (B,Hkv,d),
    sv (B,Hkv,d), following the layout the library writes (regions 256-byte aligned)."""
    torch = _torch()
    nqb, nkb = n_blocks(N)
    npad = -(-N // 64) * 64
    u8 = ws if ws.dtype == torch.uint8 else ws.view(torch.uint8)

    def take(off, nbytes):
        return u8[off:off + nbytes], off + ((nbytes + 255) // 256) * 256

    off = 0
    q8, off = take(off, B * Hq * N * d)
    k8, off = take(off, B * Hkv * N * d)
    v8, _ = take(off, B * Hkv * d * npad)
    _, off = take(off, max(B * Hkv * d * npad, 2 * B * Hkv * N * d))
    sq, off = take(off, 4 * B * Hq * nqb)
    sk, off = take(off, 4 * B * Hkv * nkb)
    km, off = take(off, 4 * B * Hkv * d)
    sv, off = take(off, 4 * B * Hkv * d)
    f = lambda t: t.view(torch.float32)
    return dict(q8=q8.view(B, Hq, N, d), k8=k8.view(B, Hkv, N, d), v8=v8.view(B, Hkv, d, npad),
                sq=f(sq).view(B, Hq, nqb), sk=f(sk).view(B, Hkv, nkb), kmean=f(km).view(B, Hkv, d),
                sv=f(sv).view(B, Hkv, d))


def block_sparse_attn(q, k, v, mask=None, lam: float = -math.inf, causal: bool = False, out=None, stats=None,
                      precision: int = SPARGE_PRECISION_BF16, ws=None):
    """Stage 2: attention over the kept 128x64 tiles with the lambda warp filter.
    precision SPARGE_PRECISION_Q8 (e4m3 Q.K^T, f16 P.V), SPARGE_PRECISION_Q8_FP8PV (both
    products e4m3) or SPARGE_PRECISION_BF16_FP8PV (bf16 Q.K^T, e4m3 P.V) runs an 8-bit path
    (d = 128); its workspace then holds the quantised copies and scales (see q8_ws_views)."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(q)
    op = SPARGE_OP_BLOCK_SPARSE_ATTN_Q8 if precision in PRECISIONS_8BIT \
        else SPARGE_OP_BLOCK_SPARSE_ATTN
    ws = _workspace(op, q, k, ws)
    dq, dk, dv, do = _desc(q), _desc(k), _desc(v), _desc(out)
    mp = 0 if mask is None else mask.data_ptr()
    sp = 0 if stats is None else stats.data_ptr()
    _check(lib().sparge_block_sparse_attn(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), mp, float(lam),
                                          int(causal), int(precision), ctypes.byref(do), ws.data_ptr(), ws.numel(),
                                          sp, _stream()))
    return out


def sparge_attn(q, k, v, topk: float = 0.5, causal: bool = False, out=None, ws=None):
    """The plug-and-play call: predicted mask (theta 0.5) then block-sparse attention."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(q)
    ws = _workspace(SPARGE_OP_ATTN, q, k, ws)
    dq, dk, dv, do = _desc(q), _desc(k), _desc(v), _desc(out)
    _check(lib().sparge_attn(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), float(topk), int(causal),
                             ctypes.byref(do), ws.data_ptr(), ws.numel(), _stream()))
    return out


def _head_array(x, name):
    """A per-head parameter array as a device pointer (0 for None); x is a float32 CUDA tensor."""
    if x is None:
        return 0
    torch = _torch()
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.float32 and x.dim() == 1
            and x.is_contiguous()):
        raise TypeError("%s must be a contiguous float32 CUDA tensor of Hq entries" % name)
    return x.data_ptr()


def _order_ptr(order):
    """A token order as a device pointer (0 for None); order is an int32 CUDA tensor of N entries."""
    if order is None:
        return 0
    torch = _torch()
    if not (isinstance(order, torch.Tensor) and order.is_cuda and order.dtype == torch.int32 and order.dim() == 1
            and order.is_contiguous()):
        raise TypeError("token_order must be a contiguous int32 CUDA tensor of N entries")
    return order.data_ptr()


def _params(theta, lam, scale, precision, stats, events, topk_h=None, theta_h=None, lam_h=None, order=None,
            topk_mode=0, topp=1.0):
    """A sparge_params; `events` (6 torch.cuda.Event or None) are passed as cudaEvent_t handles.
    The handle array is kept on the returned struct so it outlives the call.  topk_h, theta_h and
    lam_h are optional per-query-head float32 CUDA tensors; order an optional int32 token order."""
    evp = None
    if events is not None:
        assert len(events) == 6
        for ev in events:
            if not ev.cuda_event:
                ev.record()   # torch creates the event on its first record
        evp = (ctypes.c_void_p * 6)(*[ev.cuda_event for ev in events])
    p = sparge_params(float(theta), float(lam), float(scale), int(precision),
                      0 if stats is None else stats.data_ptr(),
                      ctypes.cast(evp, ctypes.c_void_p) if evp is not None else None,
                      _head_array(topk_h, "topk_per_head"), _head_array(theta_h, "theta_per_head"),
                      _head_array(lam_h, "lambda_per_head"), _order_ptr(order), int(topk_mode), float(topp))
    p._evp = evp
    p._arrays = (topk_h, theta_h, lam_h, order)
    return p


def block_sparse_attn_ex(q, k, v, mask=None, causal: bool = False, lam: float = -math.inf, scale: float = 0.0,
                         precision: int = SPARGE_PRECISION_BF16, stats=None, out=None, ws=None, events=None,
                         lambda_per_head=None, token_order=None):
    """block_sparse_attn with an explicit scale, optional timing events (6 torch.cuda.Event:
    [0] before the V copy or quantisation, [4] after it, [5] after the attention kernel) and an
    optional per-query-head lambda (float32 CUDA tensor of Hq entries) and an optional token order
    (int32 CUDA tensor of N entries; the mask then refers to the reordered sequence and the output
    comes back in the original order)."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(q)
    op = SPARGE_OP_BLOCK_SPARSE_ATTN_Q8 if precision in PRECISIONS_8BIT \
        else SPARGE_OP_BLOCK_SPARSE_ATTN
    ws = _workspace(op | (SPARGE_OP_TOKEN_ORDER if token_order is not None else 0), q, k, ws)
    p = _params(0.5, lam, scale, precision, stats, events, lam_h=lambda_per_head, order=token_order)
    dq, dk, dv, do = _desc(q), _desc(k), _desc(v), _desc(out)
    mp = 0 if mask is None else mask.data_ptr()
    _check(lib().sparge_block_sparse_attn_ex(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), mp, int(causal),
                                             ctypes.byref(p), ctypes.byref(do), ws.data_ptr(), ws.numel(), _stream()))
    return out


def sparge_attn_ex(q, k, v, topk: float, causal: bool, theta: float = 0.5, lam: float = -math.inf,
                   scale: float = 0.0, precision: int = SPARGE_PRECISION_BF16, stats=None, mask_out=None,
                   out=None, ws=None, events=None, topk_per_head=None, theta_per_head=None, lambda_per_head=None,
                   token_order=None, topk_mode: int = SPARGE_TOPK_CUMULATIVE, topp: float = 1.0):
    """sparge_attn with explicit theta, lambda, scale, counters, an optional mask output,
    optional timing events (6 torch.cuda.Event, recorded around the five kernels), optional
    per-query-head topk, theta and lambda (float32 CUDA tensors of Hq entries) and an optional
    token order (int32 CUDA tensor of N entries: blocks and mask_out refer to the reordered
    sequence, the output comes back in the original order)."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(q)
    q8 = precision in PRECISIONS_8BIT
    ws = _workspace((SPARGE_OP_ATTN_Q8 if q8 else SPARGE_OP_ATTN) | (SPARGE_OP_TOKEN_ORDER if token_order is not None else 0),
                    q, k, ws)
    p = _params(theta, lam, scale, precision, stats, events, topk_per_head, theta_per_head, lambda_per_head,
                token_order, topk_mode, topp)
    dq, dk, dv, do = _desc(q), _desc(k), _desc(v), _desc(out)
    mp = 0 if mask_out is None else mask_out.data_ptr()
    _check(lib().sparge_attn_ex(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), float(topk), int(causal),
                                ctypes.byref(p), ctypes.byref(do), mp, ws.data_ptr(), ws.numel(), _stream()))
    return out


def permute_tokens(x, perm, out=None):
    """y[:, :, t] = x[:, :, perm[t]] (perm: int32 CUDA tensor)."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(x)
    dx, dy = _desc(x), _desc(out)
    _check(lib().sparge_permute_tokens(ctypes.byref(dx), perm.data_ptr(), ctypes.byref(dy), _stream()))
    return out


def unpermute_tokens(x, perm, out=None):
    """y[:, :, perm[t]] = x[:, :, t]."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(x)
    dx, dy = _desc(x), _desc(out)
    _check(lib().sparge_unpermute_tokens(ctypes.byref(dx), perm.data_ptr(), ctypes.byref(dy), _stream()))
    return out


def window_attn(q, k, v, window: int, sinks: int = 0, scale: float = 0.0, out=None, ws=None):
    """Causal attention over each query's last `window` keys (itself included) and the first `sinks` keys; q may be
    shorter than k and v (its last query sits on the last key)."""
    return (_binding_module or _load_binding()).window_attn(q, k, v, window, sinks, scale, out, ws)


def rope_freqs(rot_dim: int, base: float = 10000.0, device="cuda"):
    """The rotation's inverse frequencies base^(-2i/rot_dim), float64, for qk_norm_rope (scaled variants: scale
    this tensor)."""
    torch = _torch()
    return base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)


def qk_norm_rope(q, k, inv_freq=None, positions=None, start: int = 0, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None):
    """Norm of q (B,Hq,N,d) and k (B,Hkv,N,d) over each head's channels, times the weights (float32, d
    entries, or None), then the rotation of the first 2 len(inv_freq) channels by the positions ((B, N) int32,
    or start, start + 1, ...); inv_freq: float64 CUDA tensor (rope_freqs) or None (norm only).  Returns (q_out,
    k_out), which may be given and may be q and k (made here, they share one storage up to 1 MB in all)."""
    return (_binding_module or _load_binding()).qk_norm_rope(q, k, inv_freq, positions, start, q_weight, k_weight, eps,
                                                        interleaved, q_out, k_out)


def rope_axes(sections, woven: bool = False, device="cuda"):
    """The axis of each rotated pair, int32, for qk_norm_rope_axes: sections[x] pairs of axis x, one axis after the other, or
    (woven) the axes taking turns pair by pair while they have pairs left."""
    torch = _torch()
    if any(n < 0 for n in sections):
        raise ValueError("sections must not be negative: %r" % (tuple(sections),))
    if woven:
        left, axes = list(sections), []
        while any(left):
            for x, n in enumerate(left):
                if n > 0:
                    left[x] = n - 1
                    axes.append(x)
    else:
        axes = [x for x, n in enumerate(sections) for _ in range(n)]
    return torch.tensor(axes, dtype=torch.int32, device=device)


def rope_grid_positions(n_prefix: int, T: int, H: int, W: int, order=None, device="cuda"):
    """Positions (3, 1, N) int32 of n_prefix text tokens and a T x H x W grid behind them (tokens row-major, as
    hilbert_perm_3d numbers them): text token i stands at i on every axis, grid token (t, y, x) at n_prefix + t, + y,
    + x.  order (int32, N entries): positions of the tokens in that order."""
    torch = _torch()
    text = torch.arange(n_prefix, dtype=torch.int32, device=device).expand(3, -1)
    grid = torch.stack(torch.meshgrid(*(torch.arange(n, dtype=torch.int32, device=device) for n in (T, H, W)), indexing="ij"))
    pos = torch.cat([text, n_prefix + grid.flatten(1)], 1)
    return (pos if order is None else pos[:, order.long()])[:, None].contiguous()


def qk_norm_rope_axes(q, k, inv_freq, axes, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, k_out=None):
    """qk_norm_rope with positions on several axes (images, video): pair i turns by positions[axes[i], b, n] *
    inv_freq[i].  positions (A, B, N) int32, A <= 4, tokens contiguous, any other strides (a batch may be expanded); axes: int32 CUDA
    tensor of as many entries as inv_freq (rope_axes)."""
    return (_binding_module or _load_binding()).qk_norm_rope_axes(q, k, inv_freq, axes, positions, q_weight, k_weight, eps,
                                                             interleaved, q_out, k_out)


def cache_tables(lens, new_lens, free_pages, table, page_size: int, N: int, slots=None, positions=None, kv_lens=None,
                 used=None):
    """Block tables and slot maps of a step: extends table (R, width; int32, rows any stride) in place with pages
    from the front of free_pages and returns (slots (R, N) int64, positions (R, N) int32, kv_lens (R) int32,
    used (1) int32); the new tokens stand right-aligned, -1 in front of them (see sparge_cache_tables).  Outputs that the
    call makes share one storage up to 64 KB in all."""
    return (_binding_module or _load_binding()).cache_tables(lens, new_lens, free_pages, table, page_size, N, slots, positions,
                                                        kv_lens, used)


def cache4_pool(n_pages: int, page_size: int, H: int, d: int, device="cuda"):
    """An empty pool of the 4-bit cache: a uint8 tensor (n_pages, H, page_size / 16, 18 d), from whose shape the
    other calls read page size, heads and head dim."""
    torch = _torch()
    if n_pages < 0 or lib().sparge_cache4_bytes(max(1, n_pages), page_size, H, d) == 0:
        raise ValueError("unsupported pool: n_pages=%d, page_size=%d, H=%d, d=%d" % (n_pages, page_size, H, d))
    return torch.zeros((n_pages, H, page_size // 16, 18 * d), dtype=torch.uint8, device=device)


def cache4_store(k, v, slots, pool):
    """Stores rows (b, h, n) of k and v (B,H,N,d) at slots[b, n] ((B, N) int64; negative: left out) of the pool."""
    (_binding_module or _load_binding()).cache4_store(k, v, slots, pool)


def cache4_load(pool, slots, k_out=None, v_out=None):
    """The rows at slots ((B, N) int64) as bf16 (B,H,N,d) tensors k and v.  Rows of left-out (negative) slots are zero
    in tensors made here (which share one storage up to 1 MB in all) and stay as they were in tensors that are given."""
    return (_binding_module or _load_binding()).cache4_load(pool, slots, k_out, v_out)


def cache4_attn(q, pool, table, kv_lens, window: int = 0, sinks: int = 0, scale: float = 0.0, out=None, ws=None):
    """Attention of q (B,Hq,Nq,d) over the 4-bit cache: sequence b has kv_lens[b] tokens on the pages table[b, :]
    ((B, width) int32) and q holds its last Nq; window > 0 keeps each query's last `window` tokens and the first
    `sinks`."""
    return (_binding_module or _load_binding()).cache4_attn(q, pool, table, kv_lens, window, sinks, scale, out, ws)


def cache4_bounds(n_pages: int, H: int, d: int, device="cuda"):
    """Bounds for a pool of n_pages pages, all zero: a uint8 tensor (n_pages, bytes of a page's bounds)."""
    torch = _torch()
    row = int(lib().sparge_cache4_bounds_bytes(1, H, d)) if H > 0 else 0
    if n_pages < 0 or row == 0:
        raise ValueError("unsupported pool: n_pages=%d, H=%d, d=%d" % (n_pages, H, d))
    return torch.zeros((n_pages, row), dtype=torch.uint8, device=device)


def cache4_bounds_update(pool, table, kv_lens, N: int, bounds):
    """Renews the bounds of the pages on which the last N of each sequence's kv_lens[b] tokens lie (after a
    cache4_store of N new ones); table ((B, width) int32) and kv_lens as cache4_attn takes them.  Of sequences that share
    a page (in the same column of table) the one with the most tokens on it counts."""
    (_binding_module or _load_binding()).cache4_bounds_update(pool, table, kv_lens, N, bounds)


def cache4_bounds_load(pool, bounds, pages):
    """The bounds of pages (int32, any shape) as values: hi and lo, bf16 of shape (pages.numel(), H, d), zero for
    negative pages."""
    return (_binding_module or _load_binding()).cache4_bounds_load(pool, bounds, pages)


def cache4_select(q, pool, bounds, table, kv_lens, keep: int, first: int = 1, last: int = 1, pages=None, lens=None,
                  ws=None):
    """For each query of q (B,Hq,Nq,d) and KV head the pages that its keys' bounds say matter most: the `first` first and the `last`
    last pages that the query sees, then the largest bounds on a product with a query of the head's group, up to keep pages.  (Bounds are
    rounded to one power of two a page and head: a page with one key far above its others ranks too high, by at most that power times sum |q|.)
    Returns (pages (B,Nq,Hkv,keep) int32, in order, -1 behind them; lens (B,Nq) int32, the tokens on them)."""
    return (_binding_module or _load_binding()).cache4_select(q, pool, bounds, table, kv_lens, keep, first, last, pages, lens,
                                                            ws)


def cache4_pages_attn(q, pool, pages, lens, scale: float = 0.0, out=None, ws=None):
    """Attention of each query over its own list of pages (from cache4_select) in every KV head."""
    return (_binding_module or _load_binding()).cache4_pages_attn(q, pool, pages, lens, scale, out, ws)


def cache4_prefix_attn(q, pool, prefix_pages, table, kv_lens, scale: float = 0.0, out=None, ws=None,
                       path: int = SPARGE_PREFIX_AUTO):
    """cache4_attn for sequences that all begin with the tokens on prefix_pages (int32): those are attended once for the whole
    batch, or, where path is SPARGE_PREFIX_AUTO and the sizes say that this takes longer, by each sequence.  The rows of table hold
    the prefix's pages too, kv_lens counts its tokens."""
    return (_binding_module or _load_binding()).cache4_prefix_attn(q, pool, prefix_pages, table, kv_lens, scale, path, out, ws)


def hilbert_perm_2d(n_prefix: int, H: int, W: int) -> np.ndarray:
    out = np.empty(n_prefix + H * W, dtype=np.int32)
    _check(lib().sparge_hilbert_perm_2d(n_prefix, H, W, out.ctypes.data))
    return out


def hilbert_perm_3d(n_prefix: int, T: int, H: int, W: int) -> np.ndarray:
    out = np.empty(n_prefix + T * H * W, dtype=np.int32)
    _check(lib().sparge_hilbert_perm_3d(n_prefix, T, H, W, out.ctypes.data))
    return out


def selftest_bounded_wait(limit_ns: int = 50_000_000):
    """Enqueue the library's bounded-wait self test (a wait that is made to run out)."""
    _check(lib().sparge_selftest_bounded_wait(int(limit_ns), _stream()))


def device_status() -> int:
    """Reads and clears the library's device status word (0 = fine)."""
    return int(lib().sparge_get_device_status(_stream()))
