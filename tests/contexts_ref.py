"""fp64 definitions of the operators for long shared and multimodal contexts, for the GPU tests: plain torch and Python, one
page or query at a time, nothing shared with the package."""
import math

import torch

import serving_ref as R


def norm_rope_axes(x, w, freq, axes, pos, eps, interleaved):
    """x (B,H,N,d) fp64, pos (A,B,N), axes a list: y and the magnitude of what was summed."""
    y, mag = R.norm_rope(x, w, None, None, eps, interleaved)
    y, mag = y.clone(), mag.clone()
    n = len(axes)
    for i, ax in enumerate(axes):
        ang = (pos[ax].double() * freq[i])[:, None]
        c, s = torch.cos(ang), torch.sin(ang)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def unit(a):
    """The least power of two s >= 2^-126 with a <= 127 s, a Python float."""
    if not math.isfinite(a):
        return math.inf
    s = 2.0 ** -126
    while a > 127.0 * s:
        s *= 2.0
    return s


def page_bounds(k):
    """k (tokens, d) fp64 of one page and head: hi, lo (d) and s."""
    if not bool(torch.isfinite(k).all()):
        inf = torch.full((k.shape[1],), math.inf, dtype=torch.float64)
        return inf, -inf, math.inf
    hi, lo = k.amax(0).cpu(), k.amin(0).cpu()
    s = unit(float(torch.maximum(hi.abs(), lo.abs()).max()))
    return torch.ceil(hi / s) * s, torch.floor(lo / s) * s, s


def scores(q, hi, lo):
    """q (G, d) fp64 bf16 values, hi and lo (pages, d): each page's score of the group."""
    best = torch.full((hi.shape[0],), -math.inf, dtype=torch.float64)
    for row in q.cpu():
        if not bool(torch.isfinite(row).all()):
            x = torch.zeros(hi.shape[0], dtype=torch.float64)
        else:
            t = unit(float(row.abs().max()))
            r = torch.round(row / t)
            fine = torch.isfinite(hi).all(-1)
            x = t * torch.maximum(r * torch.where(fine[:, None], hi, 0), r * torch.where(fine[:, None], lo, 0)).sum(-1)
        best = torch.maximum(best, x)
    return torch.where(torch.isfinite(hi).all(-1), best, math.inf)


def choose(score, keep, first, last):
    """Page numbers (ascending) of the len(score) pages that are kept."""
    n = len(score)
    if n <= keep:
        return list(range(n))
    fixed = [j for j in range(n) if j < first or j >= n - last]
    rest = sorted((j for j in range(n) if first <= j < n - last), key=lambda j: (-score[j], j))
    return sorted(fixed + rest[:keep - len(fixed)])
