"""Operators for long shared and multimodal contexts in the 4-bit cache, as measured cases.

Four operators: the norm of queries and keys with a rotation over several position axes
(``qk_norm_rope_axes``), the bounds of the cache's pages (``cache4_bounds_update`` with
``cache4_bounds_load``), the attention over pages that those bounds select for each query
(``cache4_select`` with ``cache4_pages_attn``) and the attention of a batch whose sequences begin with the
same prefix (``cache4_prefix_attn``).

``run`` computes a case in plain torch operations (fp32, fp64 for angles) when ``own`` is false and
calls the package when it is true, on the same state.  ``exact`` is the definition in fp64.

The bounds of a page and head: hi and lo of each channel over the page's tokens as the cache reads them back, in
int8 codes of a power of two s, the least that holds them (s >= 2^-126): ceil(hi / s), floor(lo / s).  A query row r
(int8 codes of a power of two t, rounded to even) scores a page with t s sum_c max(r_c hi_c, r_c lo_c); the heads of a KV
head take their largest.  Everything is a whole number times a power of two, so selections agree exactly.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

GROUP = 16    # tokens of a cache record
CHANNELS = 64  # channels that share a scale and a minimum


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _cdiv(a, b):
    return -(-a // b)


def _sections(c):
    """Pairs of each axis."""
    return [int(x) for x in c["sections"].split()]


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # the decoding step of a 32/8-head model over images and text: 64 sequences, three axes
        dict(name="axes, 64 tokens decode", op="axes", B=64, Hq=32, Hkv=8, N=1, d=128, sections="16 24 24", woven=False,
             base=500000.0, max_pos=131072, interleaved=False, weights=True),
        # the 30-head video workload: 226 text tokens and 13 frames of 30 x 45, every axis with frequencies of its own
        dict(name="axes, video 17776", op="axes", B=1, Hq=30, Hkv=30, N=17776, d=64, sections="8 12 12", woven=False,
             base=10000.0, max_pos=17776, interleaved=True, weights=True),
        # a 32K prefill of a 32/8-head model, the axes taking turns pair by pair
        dict(name="axes, prefill 32K", op="axes", B=1, Hq=32, Hkv=8, N=32768, d=128, sections="24 20 20", woven=True,
             base=500000.0, max_pos=131072, interleaved=False, weights=True),
        # a decoding step appended a token to each of 256 sequences
        dict(name="bounds, 256 appended", op="bounds", B=256, Hkv=8, N=1, d=128, page=64),
        # a prefill chunk of 8192 tokens was stored for each of four sequences
        dict(name="bounds, 4 chunks of 8192", op="bounds", B=4, Hkv=8, N=8192, d=128, page=64),
        # four answers to one prompt: latency
        dict(name="prefix, 4 over 4K", op="prefix", B=4, Hq=32, Hkv=8, Nq=1, d=128, page=64, prefix=4096, own_min=16, own_max=256),
        # a full decoding batch behind a long system prompt or video
        dict(name="prefix, 64 over 32K", op="prefix", B=64, Hq=32, Hkv=8, Nq=1, d=128, page=64, prefix=32768, own_min=64,
             own_max=2048),
        # many short requests with two speculative tokens, small heads and pages
        dict(name="prefix, 256 x 2 over 8K", op="prefix", B=256, Hq=16, Hkv=4, Nq=2, d=64, page=16, prefix=8192, own_min=19,
             own_max=1031),
        # a few users of a document of 128K tokens
        dict(name="prefix, 12 over 128K", op="prefix", B=12, Hq=32, Hkv=8, Nq=1, d=128, page=64, prefix=131072, own_min=100,
             own_max=3001),
        # one user's decoding step at 32K tokens: latency
        dict(name="pages, 1 x 32K", op="pages", B=1, Hq=32, Hkv=8, Nq=1, d=128, page=64, len_min=32768, len_max=32768, keep=64,
             first=1, last=1),
        # a decoding batch of ragged lengths, 4096 tokens of each
        dict(name="pages, 64 x up to 32K", op="pages", B=64, Hq=32, Hkv=8, Nq=1, d=128, page=64, len_min=1024, len_max=32768,
             keep=64, first=1, last=2),
        # speculative steps of four tokens over long contexts, small heads and pages
        dict(name="pages, 24 x 4 up to 128K", op="pages", B=24, Hq=16, Hkv=4, Nq=4, d=64, page=16, len_min=515,
             len_max=131072, keep=128, first=1, last=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "bounds", "prefix", "prefix", "pages", "pages"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "axes":
        B = _log_int(rng, 1, 256)
        N = min(32768, _log_int(rng, 1, max(1, 32768 * 40 // (B * (Hkv * G + Hkv)))))
        pairs = rng.choice([d // 2, d // 4, d // 2])
        cuts = sorted(rng.randint(0, pairs) for _ in range(rng.choice([1, 2, 3])))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, sections=" ".join(str(x) for x in sections), woven=rng.random() < 0.4,
                    base=rng.choice([10000.0, 500000.0]), max_pos=_log_int(rng, 2048, 1048576),
                    interleaved=rng.random() < 0.5, weights=rng.random() < 0.7)
    if op == "bounds":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, Hkv=Hkv, N=_log_int(rng, 1, max(1, min(16384, 32768 * 8 // (B * Hkv)))), d=d, page=page)
    if op == "prefix":
        B, Nq = _log_int(rng, 2, 256), rng.choice([1, 1, 1, 2, 4, 7])
        # the listed batch over 32K bounds the products, its own tokens the rest
        most = min(131072, 64 * 32 * 32768 * 128 // (B * Nq * Hkv * G * d))
        own_most = max(Nq, 64 * 8 * 2048 // (B * Hkv * _cdiv(G * Nq, 16)))
        top = min(4096, own_most)
        lo = rng.randint(Nq, max(Nq, top // 8))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, Nq=Nq, d=d, page=page, prefix=_log_int(rng, page, max(page, most)) // page * page,
                    own_min=lo, own_max=max(lo, _log_int(rng, lo, max(lo, top))))
    B, Nq = _log_int(rng, 1, 128), rng.choice([1, 1, 1, 2, 4, 7])
    top = min(131072, max(512, 64 * 16384 * 8 // (B * Hkv)))
    hi = max(Nq, _log_int(rng, 64, top))
    first, last = rng.choice([0, 1, 1, 3]), rng.choice([1, 2, 5])
    most = max(first + last, min(1024, 64 * 8 * 4096 // (B * Nq * Hkv * page * _cdiv(G, 16))))
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, Nq=Nq, d=d, page=page, len_min=rng.randint(Nq, max(Nq, hi // 2)), len_max=hi,
                keep=rng.randint(first + last, most), first=first, last=last)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed & 0x7FFFFFFFFFFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=_device())


def _spread(lo, hi, n, g):
    """n whole numbers spread evenly over lo..hi, in an order of the seed's."""
    x = torch.linspace(lo, hi, n, device=_device(), dtype=torch.float64) if n > 1 else torch.full((1,), float(hi), device=_device())
    return x.round().to(torch.int32)[torch.randperm(n, generator=g, device=_device())]


def _keys(g, *shape):
    """Key-like rows: normal values, a few channels with an offset and a larger spread."""
    x = _randn(g, *shape)
    d = shape[-1]
    ch = torch.randperm(d, generator=g, device=x.device)[: d // 16]
    x[..., ch] = 3.0 * x[..., ch] + 4.0
    return x


def _quantise(x):
    """x (..., d) fp32 of bf16 values: codes (uint8), and scale | minimum << 16 as bf16 bits, per 64 channels."""
    y = x.unflatten(-1, (-1, CHANNELS))
    m = y.amin(-1, keepdim=True)
    s = ((y.amax(-1, keepdim=True) - m) / 15.0).bfloat16().float()
    n = torch.where(s > 0, (y - m) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    n = n.round().clamp(0, 15).to(torch.uint8).flatten(-2)
    bits = lambda t: t[..., 0].bfloat16().view(torch.int16).to(torch.int32) & 0xFFFF  # noqa: E731
    return n, bits(s) | (bits(m) << 16)


def _expand(codes, words):
    scale, low = (words << 16).view(torch.float32), (words & -65536).view(torch.float32)
    return (codes.float().unflatten(-1, (-1, CHANNELS)) * scale[..., None] + low[..., None]).flatten(-2)


def _pack(kc, km, vc, vm):
    """Codes (..., 16 tokens, d) and their words (..., 16, d / 64) as cache records (..., bytes)."""
    d = kc.shape[-1]
    k = kc.unflatten(-1, (d // 32, 4, 4, 2)).transpose(-4, -3)  # token, 8-channel piece, 32-channel word, byte, nibble
    k = (k[..., 0] | (k[..., 1] << 4)).flatten(-4)
    v = vc.unflatten(-2, (2, 4, 2)).unflatten(-1, (d // 64, 4, 2, 8))  # half, pair, parity; part, tile, nibble, row
    n = v.dim()
    lead = list(range(n - 7))
    h8, c, b2, part, tile, nib, row = range(n - 7, n)
    v = v.permute(*lead, part, row, c, tile, b2, h8, nib)
    v = (v[..., 0] | (v[..., 1] << 4)).flatten(-6)
    words = lambda t: t.contiguous().view(torch.uint8).flatten(-2)  # noqa: E731
    return torch.cat([k, words(km), v, words(vm)], -1)


def _power(a):
    """The least power of two s >= 2^-126 with a <= 127 s (fp32); infinity where a is not finite."""
    m, e = torch.frexp(a)
    e = torch.where(m <= 127.0 / 128.0, e - 7, e - 6)
    e = torch.where(a > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    return torch.where(torch.isfinite(a), torch.ldexp(torch.ones_like(a), e), torch.full_like(a, math.inf))


def _bound(k, valid):
    """Codes hi, lo (int8) and s of pages k (n, H, page, d) fp32 of which the first valid[n] tokens count."""
    there = (torch.arange(k.shape[2], device=k.device)[None] < valid[:, None])[:, None, :, None]
    hi = k.masked_fill(~there, -math.inf).amax(2)
    lo = k.masked_fill(~there, math.inf).amin(2)
    s = _power(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    return torch.ceil(hi / s[..., None]).to(torch.int8), torch.floor(lo / s[..., None]).to(torch.int8), s


def _pack_bounds(hi, lo, s):
    """(n, H, d), (n, H, d), (n, H) as the rows of a bounds tensor: codes of every head, scales, padding to 32 bytes."""
    n, H, d = hi.shape
    row = torch.zeros(n, _cdiv(H * (2 * d + 4), 32) * 32, dtype=torch.uint8, device=hi.device)
    row[:, : H * 2 * d] = torch.stack([hi, lo], 2).flatten(1).view(torch.uint8)
    row[:, H * 2 * d: H * (2 * d + 4)] = s.contiguous().view(torch.uint8)
    return row


def _pool(g, n_pages, Hkv, page, d, valid=None):
    """A filled cache: n_pages pages of random tokens, every page around a point of its own; with `valid` (tokens of
    each page that count) its bounds too."""
    rec = GROUP * (d + d // 8)
    pool = torch.empty(n_pages, Hkv, page // GROUP, rec, dtype=torch.uint8, device=_device())
    rows = []
    step = max(1, (1 << 27) // (Hkv * page * d))
    for p in range(0, n_pages, step):
        n = min(step, n_pages - p)
        k = _keys(g, n, Hkv, page // GROUP, GROUP, d)
        k += 0.5 * _randn(g, n, Hkv, 1, 1, d)
        v = _randn(g, n, Hkv, page // GROUP, GROUP, d).bfloat16().float()
        kc, km = _quantise(k.bfloat16().float())
        pool[p:p + n] = _pack(kc, km, *_quantise(v))
        if valid is not None:
            rows.append(_pack_bounds(*_bound(_expand(kc, km).flatten(2, 3), valid[p:p + n])))
    return pool if valid is None else (pool, torch.cat(rows))


def _table(g, lens, page, width, ids=None):
    """Block tables of the lengths over a shuffled pool, -1 behind each sequence's last page; and the pages in all."""
    need = (lens + page - 1) // page
    total = int(need.sum())
    if ids is None:
        ids = torch.randperm(total, generator=g, device=lens.device).to(torch.int32)
    cols = torch.arange(width, device=lens.device)
    first = torch.cumsum(need, 0) - need
    at = (first[:, None] + cols[None]).clamp(max=max(0, total - 1))
    table = torch.where(cols[None] < need[:, None], ids[at], torch.full((1, 1), -1, dtype=torch.int32, device=lens.device))
    return table.to(torch.int32).contiguous(), total


def _valid_tokens(table, lens, page, total):
    """Tokens that count of each of the pool's pages."""
    have = (lens[:, None] - page * torch.arange(table.shape[1], device=lens.device)[None]).clamp(0, page)
    valid = torch.full((total,), page, dtype=torch.int64, device=lens.device)
    on = table >= 0
    valid[table[on].long()] = have[on].long()
    return valid


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    dev = _device()
    op = c["op"]
    if op == "axes":
        B, N, d, sections = c["B"], c["N"], c["d"], _sections(c)
        A, pairs = len(sections), sum(sections)
        q = (2.0 * _randn(g, B, c["Hq"], N, d)).bfloat16()
        k = _keys(g, B, c["Hkv"], N, d).bfloat16()
        # text, then rows of a grid: the first axis steps slowly, the last one fastest, all from the sequence's own start
        start = torch.randint(0, max(1, c["max_pos"] - N + 1), (1, B, 1), generator=g, device=dev)
        n = torch.arange(N, device=dev)[None, None]
        text = N // 16
        side = max(1, round((N - text) ** (1.0 / A)))
        at = [(n - text).clamp(min=0) // side ** (A - 1 - i) % (side if i else N) for i in range(A)]
        pos = torch.cat([start + torch.minimum(n, n * 0 + text) + x for x in at]).to(torch.int32).contiguous()
        if c["woven"]:
            left, axes = list(sections), []
            while len(axes) < pairs:
                for i in range(A):
                    if left[i] > 0:
                        left[i] -= 1
                        axes.append(i)
            freq = c["base"] ** (-torch.arange(pairs, dtype=torch.float64, device=dev) / pairs)
        else:
            axes = [i for i, s in enumerate(sections) for _ in range(s)]
            freq = torch.cat([c["base"] ** (-torch.arange(s, dtype=torch.float64, device=dev) / max(1, s)) for s in sections])
        w = [(1.0 + 0.3 * _randn(g, d)).contiguous() if c["weights"] else None for _ in range(2)]
        return dict(case=c, q=q, k=k, pos=pos, freq=freq, axes=torch.tensor(axes, dtype=torch.int32, device=dev), wq=w[0],
                    wk=w[1], eps=1e-6)
    B, d, P, Hkv = c["B"], c["d"], c["page"], c["Hkv"]
    if op == "bounds":
        N = c["N"]
        lens = _spread(0, P - 1, B, g) + N    # tokens already in the page that each sequence writes on, and the new ones
        table, total = _table(g, lens, P, _cdiv(P - 1 + N, P))
        pool = _pool(g, total, Hkv, P, d)
        bounds = torch.zeros(total, _cdiv(Hkv * (2 * d + 4), 32) * 32, dtype=torch.uint8, device=dev)
        return dict(case=c, pool=pool, table=table, lens=lens, bounds=bounds, pages=table.flatten())
    q = _randn(g, B, c["Hq"], c["Nq"], d).bfloat16()
    if op == "prefix":
        L = c["prefix"]
        mine = _spread(c["own_min"], c["own_max"], B, g)
        n_own = int(((mine + P - 1) // P).sum())
        ids = torch.randperm(n_own + L // P, generator=g, device=dev).to(torch.int32)
        own_table, _ = _table(g, mine, P, _cdiv(c["own_max"], P), ids[L // P:])
        prefix = ids[: L // P].contiguous()
        table = torch.cat([prefix[None].expand(B, -1), own_table], 1).contiguous()
        return dict(case=c, q=q, pool=_pool(g, n_own + L // P, Hkv, P, d), prefix=prefix, table=table, lens=mine + L)
    lens = _spread(c["len_min"], c["len_max"], B, g)
    table, total = _table(g, lens, P, _cdiv(c["len_max"], P))
    pool, bounds = _pool(g, total, Hkv, P, d, _valid_tokens(table, lens, P, total))
    return dict(case=c, q=q, pool=pool, bounds=bounds, table=table, lens=lens)


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _plain_axes(s):
    c = s["case"]
    rot = 2 * s["freq"].numel()
    ang = s["pos"].double()[s["axes"].long()].permute(1, 2, 0) * s["freq"]      # B, N, pairs
    ang = ang[:, None]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        if w is not None:
            y = y * w
        r = y[..., :rot]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., : rot // 2], r[..., rot // 2:])
        u, t = a * cos - b * sin, a * sin + b * cos
        r = torch.stack([u, t], -1).flatten(-2) if c["interleaved"] else torch.cat([u, t], -1)
        return torch.cat([r, y[..., rot:]], -1).bfloat16()

    return dict(q=one(s["q"], s["wq"]), k=one(s["k"], s["wk"]))


def _values(rec, d, sides=(0, 1)):
    """Cache records (..., bytes) as fp32 keys and values (..., 16, d)."""
    kb, mb = GROUP * d // 2, GROUP * d // 16
    k, km, v, vm = rec.split([kb, mb, kb, mb], -1)
    word = lambda w: w.contiguous().view(torch.int32).unflatten(-1, (GROUP, d // 64))  # noqa: E731
    out = []
    if 0 in sides:
        k = k.unflatten(-1, (GROUP, 4, d // 32, 4))
        out.append(_expand(torch.stack([k & 15, k >> 4], -1).transpose(-4, -3).flatten(-4), word(km)))
    if 1 in sides:
        v = v.unflatten(-1, (d // 64, 8, 4, 4, 2, 2))
        v = torch.stack([v & 15, v >> 4], -1)
        n = v.dim()
        part, row, c, tile, b2, h8, nib = range(n - 7, n)
        v = v.permute(*range(n - 7), h8, c, b2, part, tile, nib, row).flatten(-4).flatten(-4, -2)
        out.append(_expand(v, word(vm)))
    return out


def _plain_bounds(s):
    c = s["case"]
    P, H, d = c["page"], c["Hkv"], c["d"]
    lens, table, bounds = s["lens"].long(), s["table"], s["bounds"]
    col = torch.arange(table.shape[1], device=lens.device)[None]
    old = (lens - c["N"]).clamp(min=0)
    hit = (col >= old[:, None] // P) & (col * P < lens[:, None])
    pages = table[hit].long()
    k = _values(s["pool"][pages], d, (0,))[0].flatten(2, 3)
    bounds[pages] = _pack_bounds(*_bound(k, (lens[:, None] - col * P).clamp(max=P)[hit]))
    on = s["pages"] >= 0
    row = bounds[s["pages"].clamp(min=0).long()]
    codes = row[:, : H * 2 * d].view(torch.int8).view(-1, H, 2, d).float()
    scale = row[:, H * 2 * d: H * (2 * d + 4)].contiguous().view(torch.float32)[:, :, None]
    hi, lo = ((codes[:, :, i] * scale).masked_fill(~on[:, None, None], 0).bfloat16() for i in range(2))
    return dict(hi=hi, lo=lo)


def _plain_select(s):
    c, q, bounds, table, lens = s["case"], s["q"].float(), s["bounds"], s["table"], s["lens"].long()
    B, Hq, Hkv, Nq, d, P, keep = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "d", "page", "keep"))
    G, W, dev = Hq // Hkv, table.shape[1], q.device
    t = _power(q.abs().amax(-1, keepdim=True))
    r = torch.round(q / t).view(B, Hkv, G * Nq, d)
    row = bounds[table.clamp(min=0).long()]                                        # B, W, bytes
    codes = row[..., : Hkv * 2 * d].view(torch.int8).view(B, W, Hkv, 2, d)
    scale = row[..., Hkv * 2 * d: Hkv * (2 * d + 4)].contiguous().view(torch.float32).transpose(1, 2)  # B, Hkv, W
    part = lambda i: codes[:, :, :, i].permute(0, 2, 3, 1).float()  # noqa: E731
    x = torch.matmul(r.clamp(min=0), part(0)) + torch.matmul(r.clamp(max=0), part(1))  # whole numbers below 2^24
    x = x.view(B, Hkv, G, Nq, W) * t.view(B, Hkv, G, Nq, 1)
    x = torch.where(torch.isinf(scale)[:, :, None, None], scale[:, :, None, None], x * scale[:, :, None, None])
    x = x.amax(2).transpose(1, 2).double().clamp(max=1e300)                        # B, Nq, Hkv, W
    seen = (lens[:, None] - Nq + 1 + torch.arange(Nq, device=dev)[None]).clamp(min=0)
    n = ((seen + P - 1) // P)[:, :, None, None]
    col = torch.arange(W, device=dev)
    fixed = (col < c["first"]) | (col >= n - c["last"])
    x = torch.where(fixed, torch.full_like(x, math.inf), x).masked_fill(col >= n, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :keep]
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=W)
    rank = torch.arange(keep, device=dev)
    order = torch.where(rank < n, order, torch.full_like(order, W)).sort(-1)[0]
    at = order.clamp(max=W - 1)
    pages = torch.gather(table[:, None, None].expand(B, Nq, Hkv, W), 3, at)
    pages = torch.where(order < W, pages, torch.full_like(pages, -1))
    kept = n[:, :, 0, 0].clamp(max=keep)
    last = torch.where(seen > 0, (seen - 1) % P + 1, seen)
    return pages.contiguous(), torch.where(kept > 0, (kept - 1) * P + last, kept).to(torch.int32)


def _plain_pages(s):
    c, q, pool = s["case"], s["q"].float(), s["pool"]
    B, Hq, Hkv, Nq, d, P = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "d", "page"))
    G = Hq // Hkv
    pages, lens = _plain_select(s)
    head = torch.arange(Hkv, device=q.device)[None, None, :, None]
    k, v = _values(pool[pages.clamp(min=0).long(), head], d)                       # B, Nq, Hkv, keep, records, 16, d
    k, v = k.flatten(3, 5), v.flatten(3, 5)
    q = q.view(B, Hkv, G, Nq, d).permute(0, 3, 1, 2, 4)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    x = x.masked_fill(torch.arange(k.shape[3], device=q.device) >= lens[:, :, None, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(e / e.sum(-1, keepdim=True), v).permute(0, 2, 3, 1, 4)
    return dict(out=o.reshape(B, Hq, Nq, d).bfloat16(), pages=pages, lens=lens)


def _plain_prefix(s):
    c, q, pool, table, lens = s["case"], s["q"].float(), s["pool"], s["table"], s["lens"].long()
    B, Hq, Hkv, Nq, d, P, L = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "d", "page", "prefix"))
    G, dev = Hq // Hkv, q.device
    q = q.view(B, Hkv, G * Nq, d) / math.sqrt(d)
    k, v = _values(pool[s["prefix"].long()].transpose(0, 1), d)
    k, v = k.flatten(1, 3), v.flatten(1, 3)                                         # Hkv, prefix, d
    rows = q.transpose(0, 1).reshape(Hkv, B * G * Nq, d)
    x = torch.matmul(rows, k.transpose(-1, -2))
    mine = table[:, L // P:].clamp(min=0).long()
    ko, vo = _values(pool[mine].transpose(1, 2), d)
    ko, vo = ko.flatten(2, 4), vo.flatten(2, 4)                                     # B, Hkv, own tokens, d
    y = torch.matmul(q, ko.transpose(-1, -2)).view(B, Hkv, G, Nq, -1)
    pos = (lens[:, None] - Nq + torch.arange(Nq, device=dev)[None])[:, :, None]
    seen = L + torch.arange(ko.shape[2], device=dev) <= pos                         # B, Nq, own tokens
    y = y.masked_fill(~seen[:, None, None], -math.inf).view(B, Hkv, G * Nq, -1).transpose(0, 1)
    y = y.reshape(Hkv, B * G * Nq, -1)
    m = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    x, y = torch.exp(x - m), torch.exp(y - m)
    total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    o = torch.matmul(x, v).view(Hkv, B, G * Nq, d).transpose(0, 1)
    o = o + torch.matmul(y.view(Hkv, B, G * Nq, -1).transpose(0, 1), vo)
    o = o / total.view(Hkv, B, G * Nq, 1).transpose(0, 1)
    return o.reshape(B, Hq, Nq, d).bfloat16()


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"axes": _plain_axes, "bounds": _plain_bounds, "pages": _plain_pages, "prefix": _plain_prefix}[op](s)
    import free_block_sparse_gb300 as fbs
    if op == "axes":
        q, k = fbs.qk_norm_rope_axes(s["q"], s["k"], s["freq"], s["axes"], s["pos"], q_weight=s["wq"], k_weight=s["wk"],
                                     eps=s["eps"], interleaved=c["interleaved"])
        return dict(q=q, k=k)
    if op == "bounds":
        fbs.cache4_bounds_update(s["pool"], s["table"], s["lens"], c["N"], s["bounds"])
        hi, lo = fbs.cache4_bounds_load(s["pool"], s["bounds"], s["pages"])
        return dict(hi=hi, lo=lo)
    if op == "pages":
        pages, lens = fbs.cache4_select(s["q"], s["pool"], s["bounds"], s["table"], s["lens"], c["keep"], first=c["first"],
                                        last=c["last"])
        return dict(out=fbs.cache4_pages_attn(s["q"], s["pool"], pages, lens), pages=pages, lens=lens)
    return fbs.cache4_prefix_attn(s["q"], s["pool"], s["prefix"], s["table"], s["lens"])


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def _lengths(lo, hi, n):
    return [hi] if n == 1 else [round(lo + (hi - lo) * i / (n - 1)) for i in range(n)]


def work(case):
    c = case
    d, Hkv, B = c["d"], c["Hkv"], c["B"]
    if c["op"] == "axes":
        n = B * c["N"] * (c["Hq"] + Hkv) * d
        return {"bytes": 4 * n + 4 * len(_sections(c)) * B * c["N"] + 12 * sum(_sections(c)), "flops": 9 * n}
    P = c["page"]
    token = Hkv * (d + d // 8)                       # bytes of a token's keys and values
    if c["op"] == "bounds":
        lens = [x + c["N"] for x in _lengths(0, P - 1, B)]
        pages = sum(_cdiv(n, P) - (n - c["N"]) // P for n in lens)
        tok = sum(n - (n - c["N"]) // P * P for n in lens)
        # read the keys, write the bounds, read them, write the values
        return {"bytes": tok * token // 2 + 2 * pages * Hkv * (2 * d + 4) + pages * Hkv * 4 * d + 4 * (B + 2 * pages),
                "flops": 4 * tok * Hkv * d}
    rows = B * c["Hq"] * c["Nq"]
    if c["op"] == "prefix":
        mine = _lengths(c["own_min"], c["own_max"], B)
        pairs = sum(sum(c["prefix"] + n - i for i in range(c["Nq"])) for n in mine) * c["Hq"]
        return {"bytes": (c["prefix"] + sum(mine)) * token + 4 * rows * d + 4 * ((c["prefix"] + sum(mine)) // P + B),
                "flops": 4 * pairs * d}
    lens = _lengths(c["len_min"], c["len_max"], B)
    pages = sum(_cdiv(n, P) for n in lens)
    # every query's own pages (no more than there are)
    kept = sum(min(c["Nq"] * c["keep"], _cdiv(n, P)) for n in lens)
    pairs = sum(c["Nq"] * min(c["keep"] * P, n) for n in lens) * c["Hq"]
    return {"bytes": pages * (Hkv * (2 * d + 4) + 4) + kept * P * token + 4 * rows * d + 4 * c["Nq"] * (kept * Hkv + B),
            "flops": 4 * pairs * d + 2 * c["Nq"] * pages * c["Hq"] * d}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_records(rec, d):
    """Keys and values (..., 16, d) in fp64 of records (..., bytes), byte and shift of each channel looked up."""
    dev = rec.device
    t = torch.arange(GROUP, device=dev)[:, None]
    i = torch.arange(d, device=dev)[None]
    kb = t * (d // 2) + (i % 32 // 8) * (d // 8) + (i // 32) * 4 + i % 8 // 2
    ks = (i % 2) * 4 + 0 * t
    vb = (i // 64) * 512 + ((i % 8) * 4 + t % 8 // 2) * 16 + (i % 64 // 16) * 4 + (t % 2) * 2 + t // 8
    vs = (i % 16 // 8) * 4 + 0 * t
    kv, half = [], GROUP * (d // 2 + d // 16)
    for base, byte, shift in ((0, kb, ks), (half, vb, vs)):
        code = ((rec[..., base + byte.flatten()].int() >> shift.flatten().int()) & 15).double()
        w = rec[..., base + GROUP * d // 2: base + half].long().unflatten(-1, (GROUP, d // 64, 2, 2))
        f = ((w[..., 0] + 256 * w[..., 1]).to(torch.int32) << 16).view(torch.float32).double()
        f = f.repeat_interleave(CHANNELS, -2)            # record's token, channel, (scale, minimum)
        kv.append(code.unflatten(-1, (GROUP, d)) * f[..., 0] + f[..., 1])
    return kv


def _exact_power(a):
    """As a Python loop over the logarithm's neighbours would: the least power of two >= a / 127, at least 2^-126."""
    x = a.double().clamp(min=1e-300) / 127.0
    e = torch.floor(torch.log2(x))
    e = torch.where(torch.exp2(e - 1) >= x, e - 1, torch.where(torch.exp2(e) >= x, e, torch.where(torch.exp2(e + 1) >= x, e + 1, e + 2)))
    return torch.exp2(e.clamp(min=-126))


def _exact_attention(q, k, v, limit):
    """q (Hkv, G, n, d) sees tokens of k and v (Hkv, L, d) below limit (n), all fp64."""
    x = torch.einsum("hgnd,hld->hgnl", q, k) * q.shape[-1] ** -0.5
    hidden = torch.arange(k.shape[1], device=q.device)[None] >= limit[:, None]
    return torch.einsum("hgnl,hld->hgnd", torch.softmax(x.masked_fill(hidden, -math.inf), -1), v)


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    d = c["d"]
    if c["op"] == "axes":
        rot = 2 * s["freq"].numel()
        ang = torch.einsum("abn,pa->bnp", s["pos"].double(), torch.nn.functional.one_hot(s["axes"].long(), len(_sections(c))).double()
                           * s["freq"][:, None])
        turn = torch.polar(torch.ones_like(ang), ang)[:, None]

        def one(x, w):
            y = x.double()
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + s["eps"])
            y = y if w is None else y * w.double()
            lo, hi = y[..., :rot], y[..., rot:]
            z = lo.unflatten(-1, (-1, 2)) if c["interleaved"] else lo.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat([z, hi], -1)

        return dict(q=one(s["q"], s["wq"]), k=one(s["k"], s["wk"]))
    B, P, Hkv = c["B"], c["page"], c["Hkv"]
    lens = s["lens"].tolist()
    if c["op"] == "bounds":
        out = {n: torch.zeros(B, s["table"].shape[1], Hkv, d, dtype=torch.float64, device=s["lens"].device) for n in ("hi", "lo")}
        for b in range(B):
            n = _cdiv(lens[b], P)                        # every page of a sequence holds new tokens
            k = _exact_records(s["pool"][s["table"][b, :n].long()], d)[0].flatten(2, 3)     # n, Hkv, P, d
            last = lens[b] - (n - 1) * P
            for name, f, far in (("hi", torch.amax, -math.inf), ("lo", torch.amin, math.inf)):
                x = k.clone()
                x[-1, :, last:] = far
                out[name][b, :n] = f(x, 2)
            h, l = out["hi"][b, :n], out["lo"][b, :n]
            u = _exact_power(torch.maximum(h, -l).amax(-1, keepdim=True))
            out["hi"][b, :n], out["lo"][b, :n] = torch.ceil(h / u) * u, torch.floor(l / u) * u
        return {n: x.flatten(0, 1) for n, x in out.items()}
    Nq, G = c["Nq"], c["Hq"] // Hkv
    q = s["q"].double().view(B, Hkv, G, Nq, d)
    out = torch.zeros_like(q)
    if c["op"] == "prefix":
        if 1.5e-12 * B * c["Hq"] * Nq * c["prefix"] * d * 4 > 12:   # seconds at about 0.7 TFLOP/s of fp64
            return None
        base = _exact_records(s["pool"][s["prefix"].long()], d)
        base = [x.transpose(0, 1).flatten(1, 3) for x in base]
        for b in range(B):
            pages = s["table"][b, c["prefix"] // P: _cdiv(lens[b], P)].long()
            tail = [x.transpose(0, 1).flatten(1, 3) for x in _exact_records(s["pool"][pages], d)]
            k, v = (torch.cat(x, 1) for x in zip(base, tail))
            out[b] = _exact_attention(q[b], k, v, lens[b] - Nq + 1 + torch.arange(Nq, device=q.device))
        return out.view(s["q"].shape)
    # pages: chosen for one query and KV head after another
    r = q.abs().amax(-1, keepdim=True)
    t = _exact_power(r)
    r = torch.round(q / t).to(torch.int16)
    pages = np.full((B, Nq, Hkv, c["keep"]), -1, dtype=np.int32)
    kept_len = np.zeros((B, Nq), dtype=np.int32)
    for b in range(B):
        n_all = _cdiv(lens[b], P)
        ids = s["table"][b, :n_all].long()
        row = s["bounds"][ids]
        code = row[:, : Hkv * 2 * d].view(torch.int8).view(n_all, Hkv, 2, d).to(torch.int16)
        unit = row[:, Hkv * 2 * d: Hkv * (2 * d + 4)].contiguous().view(torch.float32).double()
        ids = ids.cpu().numpy()
        for i in range(Nq):
            seen = lens[b] - Nq + 1 + i
            n = _cdiv(seen, P)
            if n <= 0:
                continue
            m = min(n, c["keep"])
            kept_len[b, i] = (m - 1) * P + (seen - 1) % P + 1
            for h in range(Hkv):
                score = None
                for j in range(G):
                    x = torch.maximum(code[:n, h, 0] * r[b, h, j, i], code[:n, h, 1] * r[b, h, j, i]).sum(-1).double()
                    x = x * t[b, h, j, i] * unit[:n, h]
                    score = x if score is None else torch.maximum(score, x)
                col = np.arange(n)
                free = ~((col < c["first"]) | (col >= n - c["last"]))
                at = np.sort(np.lexsort((col, -score.cpu().numpy(), free))[:m])
                pages[b, i, h, :m] = ids[at]
                rec = s["pool"][torch.from_numpy(ids[at]).to(q.device), h]
                k, v = (x.flatten(0, 1).flatten(0, 1)[None] if x.dim() == 4 else x.flatten(0, 1)[None] for x in _exact_records(rec, d))
                out[b, h:h + 1, :, i:i + 1] = _exact_attention(q[b, h:h + 1, :, i:i + 1], k, v, torch.tensor([kept_len[b, i]], device=q.device))
    dev = q.device
    return dict(out=out.view(s["q"].shape), pages=torch.from_numpy(pages).to(dev), lens=torch.from_numpy(kept_len).to(dev))
