"""fp64 definitions of the serving operators, for the GPU tests: plain torch, one token at a time where
that is clearer, nothing shared with the package."""
import math

import torch


def norm_rope(x, w, freq, pos, eps, interleaved):
    """x (B,H,N,d) fp64; pos (B,N); freq (rot/2) fp64 or None.  Returns y and the magnitude of what was summed."""
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    mag = y.abs()
    if freq is not None and freq.numel():
        h = freq.numel()
        ang = pos.double()[:, None, :, None] * freq
        c, s = torch.cos(ang), torch.sin(ang)
        ia = torch.arange(h, device=x.device) * 2 if interleaved else torch.arange(h, device=x.device)
        ib = ia + (1 if interleaved else h)
        a, b = y[..., ia], y[..., ib]
        y, mag = y.clone(), mag.clone()
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def quantise(x):
    """Codes, scales and minima of x (..., d) fp64 (bf16 values), per 64 channels."""
    g = x.unflatten(-1, (-1, 64))
    m = g.amin(-1, keepdim=True)
    s = ((g.amax(-1, keepdim=True) - m) / 15).float().bfloat16().double()
    n = torch.where(s > 0, torch.round((g - m) / torch.where(s > 0, s, 1.0)).clamp(0, 15), torch.zeros_like(g))
    bad = ~torch.isfinite(g).all(-1, keepdim=True)
    n, s, m = (torch.where(bad, v, t) for t, v in ((n, torch.zeros_like(n)), (s, torch.full_like(s, math.nan)), (m, torch.full_like(m, math.nan))))
    return n.flatten(-2), s[..., 0], m[..., 0]


def dequantise(n, s, m):
    return (n.unflatten(-1, (-1, 64)) * s[..., None] + m[..., None]).flatten(-2)


def k_place(t, i, d):
    """Byte in a record and nibble of K channel i of token t."""
    w, c, j = i // 32, i % 32 // 8, i % 8
    return t * (d // 2) + c * (d // 8) + 4 * w + j // 2, j % 2


def v_place(t, i, d):
    p, u, y, g = i // 64, i % 64 // 16, i % 16 // 8, i % 8
    return 512 * p + 16 * (4 * g + (t % 8) // 2) + 4 * u + 2 * (t % 2) + t // 8, y


def _maps(d, place, device):
    b = torch.tensor([[place(t, i, d)[0] for i in range(d)] for t in range(16)], device=device)
    y = torch.tensor([[place(t, i, d)[1] for i in range(d)] for t in range(16)], device=device)
    return b, y


def read_pool(pool, d):
    """Everything a pool holds: codes, scale, minimum of K and V, each (pages, H, page_size, ...) fp64."""
    out = []
    for base, place in ((0, k_place), (9 * d, v_place)):
        b, y = _maps(d, place, pool.device)
        n = (pool[..., base + b.flatten()].long() >> (4 * y.flatten())) & 15
        w = pool[..., base + 8 * d: base + 9 * d].long().unflatten(-1, (16, d // 64, 4))
        bits = lambda lo: ((w[..., lo] + 256 * w[..., lo + 1]).to(torch.int32) << 16).view(torch.float32).double()  # noqa: E731
        out += [n.unflatten(-1, (16, d)).flatten(2, 3).double(), bits(0).flatten(2, 3), bits(2).flatten(2, 3)]
    return out


def attention(q, k, v, pos, window, sinks, scale, extra=None):
    """q (Hq,n,d), k and v (Hkv,L,d) fp64, pos (n).  Returns (o, a, x): o zero where nothing is seen, a = sum of
    P |extra| (extra: (Hkv,L,d), what P multiplies) and x = the largest sum |q||k| scale of a row."""
    Hq, n, d = q.shape
    Hkv, L = k.shape[:2]
    tok = torch.arange(L, device=q.device)
    seen = tok[None] <= pos[:, None]
    if window:
        seen &= (tok[None] > pos[:, None] - window) | (tok[None] < sinks)
    qg = q.view(Hkv, Hq // Hkv, n, d)
    x = torch.einsum("hgnd,hld->hgnl", qg, k) * scale
    x = x.masked_fill(~seen, -math.inf)
    p = torch.softmax(x, -1)
    p = torch.where(seen.any(-1)[:, None], p, torch.zeros_like(p))
    k0, v0 = torch.nan_to_num(k), torch.nan_to_num(v)
    o = torch.einsum("hgnl,hld->hgnd", p, v0)
    a = torch.einsum("hgnl,hld->hgnd", p, (v0 if extra is None else torch.nan_to_num(extra)).abs())
    big = (torch.einsum("hgnd,hld->hgnl", qg.abs(), k0.abs()) * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
    return o.reshape(Hq, n, d), a.reshape(Hq, n, d), big.reshape(Hq, n, 1)
