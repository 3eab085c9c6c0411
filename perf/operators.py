"""The serving operators around the sparse attention, as measured cases.

Five operators: the block tables and slot maps of a paged cache (``cache_tables``), the norm and
rotation of queries and keys (``qk_norm_rope``), the 4-bit cache's store and read-back
(``cache4_store`` with ``cache4_load``), the attention that reads that cache (``cache4_attn``) and the
causal attention over a sliding window with a few first tokens (``window_attn``).

``run`` computes a case in plain torch operations (fp32, fp64 for angles) when ``own`` is false and
calls the package when it is true, on the same state.  ``exact`` is the definition in fp64.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 16    # tokens of a cache record
CHANNELS = 64  # channels that share a scale and a minimum


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # a decoding step of 256 requests: one new token each, tables of up to 32K tokens in 64-token pages
        dict(name="tables, 256 requests decode", op="tables", R=256, N=1, page=64, max_len=32768, new_min=1),
        # a prefill step of 64 requests with chunks of up to 4096 tokens in 16-token pages
        dict(name="tables, 64 chunks of 4096", op="tables", R=64, N=4096, page=16, max_len=32768, new_min=1024),
        # the decoding step of a 32/8-head model, 64 sequences at positions of their own
        dict(name="norm rope, 64 tokens decode", op="norm_rope", B=64, Hq=32, Hkv=8, N=1, d=128, rot=128,
             base=500000.0, max_pos=131072, interleaved=False, weights=True),
        # the 24-head image workload's joint sequence (512 + 64 x 64 tokens), neighbouring pairs rotated
        dict(name="norm rope, image 4608", op="norm_rope", B=1, Hq=24, Hkv=24, N=4608, d=128, rot=128,
             base=10000.0, max_pos=4608, interleaved=True, weights=True),
        # the prefill of the 32K Llama-like workload
        dict(name="norm rope, prefill 32K", op="norm_rope", B=1, Hq=32, Hkv=8, N=32768, d=128, rot=128,
             base=500000.0, max_pos=131072, interleaved=False, weights=True),
        # a decoding step appends a token to each of 256 sequences
        dict(name="cache store, 256 appended", op="store", B=256, Hkv=8, N=1, d=128, page=64),
        # a prefill chunk of 8192 tokens for each of four sequences, stored and read back for attention
        dict(name="cache store, 4 chunks of 8192", op="store", B=4, Hkv=8, N=8192, d=128, page=64),
        # one user's decoding step at 4K tokens: latency
        dict(name="cache attn, 1 x 4K", op="cache_attn", B=1, Hq=32, Hkv=8, Nq=1, d=128, page=64,
             len_min=4096, len_max=4096, window=0, sinks=0),
        # a full decoding batch of ragged lengths
        dict(name="cache attn, 64 x up to 32K", op="cache_attn", B=64, Hq=32, Hkv=8, Nq=1, d=128, page=64,
             len_min=1024, len_max=32768, window=0, sinks=0),
        # speculative steps of four tokens under a window with first tokens, small heads, small pages
        dict(name="cache attn, 128 x 4 window 4096", op="cache_attn", B=128, Hq=16, Hkv=4, Nq=4, d=64, page=16,
             len_min=515, len_max=32768, window=4096, sinks=4),
        # a decoding step of 16 sequences over a window of 8192 of 32K keys
        dict(name="window attn, 16 x 1 decode", op="window", B=16, Hq=32, Hkv=8, Nq=1, Nk=32768, d=128,
             window=8192, sinks=4),
        # the 32K Llama-like prefill under a window of 4096
        dict(name="window attn, prefill 32K", op="window", B=1, Hq=32, Hkv=8, Nq=32768, Nk=32768, d=128,
             window=4096, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "norm_rope", "store", "cache_attn", "cache_attn", "window", "window"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "tables":
        R = _log_int(rng, 1, 1024)
        N = _log_int(rng, 1, max(1, min(4096, 262144 // R)))
        return dict(op=op, R=R, N=N, page=rng.choice([16, 32, 64, 128]), max_len=_log_int(rng, 64, 65536),
                    new_min=rng.randint(0, N))
    if op == "norm_rope":
        B = _log_int(rng, 1, 256)
        N = _log_int(rng, 1, max(1, 32768 * 40 // (B * (Hkv * G + Hkv))))
        N = min(N, 32768)
        rot = rng.choice([d, d // 2, d])
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, N=N, d=d, rot=rot, base=rng.choice([10000.0, 500000.0]),
                    max_pos=_log_int(rng, 2048, 1048576), interleaved=rng.random() < 0.5, weights=rng.random() < 0.7)
    if op == "store":
        B = _log_int(rng, 1, 256)
        N = _log_int(rng, 1, max(1, min(16384, 32768 * 8 // (B * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, N=N, d=d, page=rng.choice([16, 32, 64, 128]))
    if op == "cache_attn":
        B = _log_int(rng, 1, 128)
        Nq = rng.choice([1, 1, 1, 2, 4, 7])
        top = min(131072, max(512, 64 * 16384 * 8 // (B * Hkv * _cdiv(G * Nq, 16))))
        hi = _log_int(rng, 64, top)
        windowed = rng.random() < 0.4
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, Nq=Nq, d=d, page=rng.choice([16, 32, 64, 128]),
                    len_min=rng.randint(Nq, max(Nq, hi // 2)), len_max=max(Nq, hi),
                    window=_log_int(rng, 32, 8192) if windowed else 0, sinks=rng.choice([0, 1, 4, 37]) if windowed else 0)
    B = rng.choice([1, 1, 2, 4])
    window = _log_int(rng, 64, 8192)
    if rng.random() < 0.4:
        Nq = rng.choice([1, 1, 2, 5, 8])
        Nk = _log_int(rng, 256, 131072 // B)
    else:
        # a pass costs about B Hq Nq (window + 128) pairs; the listed prefill bounds it
        most = 32 * 32768 * 4096 // (B * Hkv * G * (window + 1024))
        Nq = _log_int(rng, 64, max(65, min(32768, most)))
        Nk = Nq + (0 if rng.random() < 0.5 else _log_int(rng, 1, 32768))
    return dict(op="window", B=B, Hq=Hkv * G, Hkv=Hkv, Nq=Nq, Nk=max(Nq, Nk), d=d, window=window,
                sinks=rng.choice([0, 1, 4, 64, 100]))


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


def _pool(g, n_pages, Hkv, page, d):
    """A filled cache: n_pages pages of random tokens."""
    rec = GROUP * (d + d // 8)
    pool = torch.empty(n_pages, Hkv, page // GROUP, rec, dtype=torch.uint8, device=_device())
    step = max(1, (1 << 27) // (Hkv * page * d))
    for p in range(0, n_pages, step):
        n = min(step, n_pages - p)
        k = _keys(g, n, Hkv, page // GROUP, GROUP, d).bfloat16().float()
        v = _randn(g, n, Hkv, page // GROUP, GROUP, d).bfloat16().float()
        pool[p:p + n] = _pack(*_quantise(k), *_quantise(v))
    return pool


def _table(g, lens, page, width, spare=0):
    """Block tables of the lengths over a shuffled pool, -1 behind each sequence's last page; then the pages left."""
    need = (lens + page - 1) // page
    total = int(need.sum())
    ids = torch.randperm(total + spare, generator=g, device=lens.device).to(torch.int32)
    cols = torch.arange(width, device=lens.device)
    first = torch.cumsum(need, 0) - need
    at = (first[:, None] + cols[None]).clamp(max=max(0, total - 1))
    table = torch.where(cols[None] < need[:, None], ids[at] if total else torch.zeros_like(at, dtype=torch.int32),
                        torch.full((1, 1), -1, dtype=torch.int32, device=lens.device))
    return table.to(torch.int32).contiguous(), ids[total:].contiguous(), total


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    dev = _device()
    op = c["op"]
    if op == "tables":
        R, N, P = c["R"], c["N"], c["page"]
        lens = _spread(0, c["max_len"], R, g)
        new = _spread(min(c["new_min"], N), N, R, g)
        width = _cdiv(c["max_len"] + N, P)
        table, free, _ = _table(g, lens, P, width, spare=R * (_cdiv(N, P) + 1))
        return dict(case=c, lens=lens, new=new, table=table, free=free)
    if op == "norm_rope":
        B, N, d = c["B"], c["N"], c["d"]
        q = (2.0 * _randn(g, B, c["Hq"], N, d)).bfloat16()
        k = _keys(g, B, c["Hkv"], N, d).bfloat16()
        pos = torch.randint(0, max(1, c["max_pos"] - N + 1), (B, 1), generator=g, device=dev)
        pos = (pos + torch.arange(N, device=dev)[None]).to(torch.int32).contiguous()
        freq = c["base"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        w = [(1.0 + 0.3 * _randn(g, d)).contiguous() if c["weights"] else None for _ in range(2)]
        return dict(case=c, q=q, k=k, pos=pos, freq=freq, wq=w[0], wk=w[1], eps=1e-6)
    if op == "store":
        B, N, d, P, Hkv = c["B"], c["N"], c["d"], c["page"], c["Hkv"]
        k = _keys(g, B, Hkv, N, d).bfloat16()
        v = _randn(g, B, Hkv, N, d).bfloat16()
        before = _spread(0, P - 1, B, g)  # tokens already in the page that each sequence writes on
        per = _cdiv(P - 1 + N, P)
        pages = torch.randperm(B * per + 3, generator=g, device=dev)[: B * per].view(B, per)
        at = before[:, None].long() + torch.arange(N, device=dev)[None]
        slots = (torch.gather(pages, 1, at // P) * P + at % P).contiguous()
        pool = torch.zeros(B * per + 3, Hkv, P // GROUP, GROUP * (d + d // 8), dtype=torch.uint8, device=dev)
        return dict(case=c, k=k, v=v, slots=slots, pool=pool)
    if op == "cache_attn":
        B, d, P, Hkv = c["B"], c["d"], c["page"], c["Hkv"]
        lens = _spread(c["len_min"], c["len_max"], B, g)
        table, _, total = _table(g, lens, P, _cdiv(c["len_max"], P))
        pool = _pool(g, total, Hkv, P, d)
        q = _randn(g, B, c["Hq"], c["Nq"], d).bfloat16()
        return dict(case=c, q=q, pool=pool, table=table, lens=lens)
    B, d = c["B"], c["d"]
    q = _randn(g, B, c["Hq"], c["Nq"], d).bfloat16()
    k = _keys(g, B, c["Hkv"], c["Nk"], d).bfloat16()
    k[:, :, : c["sinks"]] *= 2.0
    v = _randn(g, B, c["Hkv"], c["Nk"], d).bfloat16()
    return dict(case=c, q=q, k=k, v=v)


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _plain_tables(s):
    c, lens, new, table, free = s["case"], s["lens"].long(), s["new"].long(), s["table"], s["free"]
    N, P, W = c["N"], c["page"], table.shape[1]
    have, total = (lens + P - 1) // P, lens + new
    need = (total + P - 1) // P - have
    first = torch.cumsum(need, 0) - need
    cols = torch.arange(W, device=lens.device)[None]
    nth = cols - have[:, None]
    fresh = (nth >= 0) & (nth < need[:, None])
    at = (first[:, None] + nth).clamp(0, max(0, free.numel() - 1))
    out = torch.where(fresh, free[at], table)
    pos = lens[:, None] + torch.arange(N, device=lens.device)[None] - (N - new)[:, None]
    there = pos >= lens[:, None]
    page = torch.gather(out, 1, (pos.clamp(min=0) // P).clamp(max=W - 1)).long()
    slots = torch.where(there, page * P + pos.clamp(min=0) % P, torch.full_like(pos, -1))
    return dict(table=out, slots=slots, positions=torch.where(there, pos, torch.full_like(pos, -1)).to(torch.int32),
                kv_lens=total.to(torch.int32), used=need.sum().to(torch.int32).view(1))


def _plain_norm_rope(s):
    c = s["case"]
    rot = c["rot"]
    ang = s["pos"].double()[:, None, :, None] * s["freq"]
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


def _plain_store(s):
    def one(x):
        n, w = _quantise(x.float())
        scale = (w << 16).view(torch.float32)
        low = (w & -65536).view(torch.float32)
        y = n.float().unflatten(-1, (-1, CHANNELS)) * scale[..., None] + low[..., None]
        return y.flatten(-2).bfloat16()

    return dict(k=one(s["k"]), v=one(s["v"]))


def _values(rec, d):
    """Cache records (..., bytes) as fp32 keys and values (..., 16, d)."""
    kb, mb = GROUP * d // 2, GROUP * d // 16
    k, km, v, vm = rec.split([kb, mb, kb, mb], -1)
    k = k.unflatten(-1, (GROUP, 4, d // 32, 4))
    k = torch.stack([k & 15, k >> 4], -1).transpose(-4, -3).flatten(-4)
    v = v.unflatten(-1, (d // 64, 8, 4, 4, 2, 2))
    v = torch.stack([v & 15, v >> 4], -1)
    n = v.dim()
    part, row, c, tile, b2, h8, nib = range(n - 7, n)
    v = v.permute(*range(n - 7), h8, c, b2, part, tile, nib, row).flatten(-4).flatten(-4, -2)

    def one(codes, words):
        w = words.contiguous().view(torch.int32).unflatten(-1, (GROUP, d // 64))
        scale, low = (w << 16).view(torch.float32), (w & -65536).view(torch.float32)
        return (codes.float().unflatten(-1, (-1, CHANNELS)) * scale[..., None] + low[..., None]).flatten(-2)

    return one(k, km), one(v, vm)


def _plain_cache_attn(s):
    c, q, pool, table, lens = s["case"], s["q"], s["pool"], s["table"], s["lens"].long()
    B, Hq, Hkv, Nq, d, P = c["B"], c["Hq"], c["Hkv"], c["Nq"], c["d"], c["page"]
    W, S, G = c["window"], c["sinks"], c["Hq"] // c["Hkv"]
    dev = q.device
    per = P // GROUP
    if W:  # the records of the first tokens, then those of the window
        ns = _cdiv(S, GROUP)
        start = (lens - Nq - W + 1).clamp(min=0) // GROUP
        win = start[:, None] + torch.arange(_cdiv(W + Nq - 1, GROUP) + 1, device=dev)[None]
        grp = torch.cat([torch.arange(ns, device=dev)[None].expand(B, ns), torch.where(win < ns, torch.full_like(win, 1 << 40), win)], 1)
    else:
        grp = torch.arange(_cdiv(c["len_max"], GROUP), device=dev)[None].expand(B, -1)
    there = grp * GROUP < lens[:, None]
    safe = torch.where(there, grp, torch.zeros_like(grp))
    page = torch.gather(table, 1, safe // per).long()
    rec = pool[page, :, safe % per]                     # B, L, Hkv, bytes
    k, v = _values(rec.transpose(1, 2), d)
    k, v = k.flatten(2, 3), v.flatten(2, 3)             # B, Hkv, tokens, d
    tok = torch.where(there, grp, torch.full_like(grp, 1 << 40))[..., None] * GROUP + torch.arange(GROUP, device=dev)
    tok = tok.flatten(1)[:, None, :]                    # B, 1, tokens
    pos = (lens[:, None] - Nq + torch.arange(Nq, device=dev)[None])[:, :, None]
    seen = tok <= pos
    if W:
        seen = seen & ((tok > pos - W) | (tok < S))
    x = torch.matmul(q.float().view(B, Hkv, G * Nq, d), k.transpose(-1, -2)) / math.sqrt(d)
    x = x.view(B, Hkv, G, Nq, -1).masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul((e / e.sum(-1, keepdim=True)).view(B, Hkv, G * Nq, -1), v)
    return o.view(B, Hq, Nq, d).bfloat16()


def _plain_window(s):
    c = s["case"]
    B, Hq, Hkv, Nq, Nk, d, W, S = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk", "d", "window", "sinks"))
    G, off, dev = Hq // Hkv, Nk - Nq, s["q"].device
    n = min(Nq, max(128, min(W, 1024)))                 # queries of a block, which share a stretch of keys
    nb = _cdiv(Nq, n)
    q = torch.nn.functional.pad(s["q"].float(), (0, 0, 0, nb * n - Nq)).view(B, Hkv, G, nb, n, d)
    q = q.transpose(2, 3).reshape(B, Hkv, nb, G * n, d)
    pos = off + torch.arange(nb * n, device=dev).view(nb, n)
    key = pos[:, :1] - W + 1 + torch.arange(n + W - 1, device=dev)[None]      # nb, L
    at = key.clamp(0, Nk - 1)
    k, v = s["k"].float(), s["v"].float()
    near = (key[:, None] >= 0) & (key[:, None] < Nk) & (key[:, None] <= pos[:, :, None]) & (key[:, None] > pos[:, :, None] - W)
    x = torch.matmul(q, k[:, :, at].transpose(-1, -2)).view(B, Hkv, nb, G, n, -1)
    x = (x / math.sqrt(d)).masked_fill(~near[:, None], -math.inf)
    first = torch.arange(min(S, Nk), device=dev)
    far = first[None, None] <= pos[:, :, None] - W
    y = torch.matmul(q, k[:, :, None, : min(S, Nk)].transpose(-1, -2)).view(B, Hkv, nb, G, n, -1)
    y = (y / math.sqrt(d)).masked_fill(~far[:, None], -math.inf)
    m = torch.cat([x.amax(-1, keepdim=True), y], -1).amax(-1, keepdim=True)
    x, y = torch.exp(x - m), torch.exp(y - m)
    total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, nb, G * n, -1), v[:, :, at]) + torch.matmul(y.reshape(B, Hkv, nb, G * n, -1), v[:, :, None, : min(S, Nk)])
    o = (o / total.view(B, Hkv, nb, G * n, 1)).view(B, Hkv, nb, G, n, d).transpose(2, 3)
    return o.reshape(B, Hq, nb * n, d)[:, :, :Nq].bfloat16()


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"tables": _plain_tables, "norm_rope": _plain_norm_rope, "store": _plain_store,
                "cache_attn": _plain_cache_attn, "window": _plain_window}[op](s)
    import free_block_sparse_gb300 as fbs
    if op == "tables":
        # the call extends the tables in place; each pass starts from the step's own
        table = s["table"].clone()
        slots, pos, kv_lens, used = fbs.cache_tables(s["lens"], s["new"], s["free"], table, c["page"], c["N"])
        return dict(table=table, slots=slots, positions=pos, kv_lens=kv_lens, used=used)
    if op == "norm_rope":
        q, k = fbs.qk_norm_rope(s["q"], s["k"], s["freq"], positions=s["pos"], q_weight=s["wq"], k_weight=s["wk"],
                                eps=s["eps"], interleaved=c["interleaved"])
        return dict(q=q, k=k)
    if op == "store":
        fbs.cache4_store(s["k"], s["v"], s["slots"], s["pool"])
        k, v = fbs.cache4_load(s["pool"], s["slots"])
        return dict(k=k, v=v)
    if op == "cache_attn":
        return fbs.cache4_attn(s["q"], s["pool"], s["table"], s["lens"], window=c["window"], sinks=c["sinks"])
    return fbs.window_attn(s["q"], s["k"], s["v"], c["window"], c["sinks"])


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def _pairs(first, n, W, S):
    """Visible (query, key) pairs of n queries at positions first, first + 1, ... ."""
    tot = 0
    for p in ([first, first + n - 1] if n > 1 else [first]):
        seen = p + 1 if not W else min(p + 1, W + min(S, max(0, p + 1 - W)))
        tot += seen
    if n <= 2:
        return tot
    if W and first >= W + S:
        return n * (W + S)
    full = n * first + n * (n + 1) // 2                  # without the window
    if not W or first + n <= W:
        return full
    hid = 0                                              # keys between the first tokens and the window
    a = max(first, W + S)
    b = first + n - 1
    if b >= a:
        m = b - a + 1
        hid = m * (a - W - S + 1) + m * (m - 1) // 2
    return full - hid


def _visible(length, Nq, W, S):
    return length if not W else min(length, W + Nq - 1 + min(S, max(0, length - W - Nq + 1)))


def _lengths(case):
    lo, hi, n = case["len_min"], case["len_max"], case["B"]
    return [hi] if n == 1 else [round(lo + (hi - lo) * i / (n - 1)) for i in range(n)]


def work(case):
    c = case
    if c["op"] == "tables":
        R, N, P = c["R"], c["N"], c["page"]
        pages = R * (c["new_min"] + N) // 2 // P
        old = R  # the page that each request's first new token falls on
        return {"bytes": 8 * R + 4 * old + 8 * pages + (8 + 4) * R * N + 4 * R + 4, "flops": 0}
    if c["op"] == "norm_rope":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return {"bytes": 4 * n + 4 * c["B"] * c["N"] + 4 * c["rot"], "flops": 9 * n}
    if c["op"] == "store":
        n = 2 * c["B"] * c["N"] * c["Hkv"] * c["d"]       # keys and values
        # read the rows, write the cache, read it, write the rows
        return {"bytes": 2 * n + 2 * (n // 2 + n // 16) + 2 * n + 16 * c["B"] * c["N"], "flops": 8 * n}
    if c["op"] == "cache_attn":
        lens = _lengths(c)
        tok = sum(_visible(n, c["Nq"], c["window"], c["sinks"]) for n in lens)
        pairs = sum(_pairs(n - c["Nq"], c["Nq"], c["window"], c["sinks"]) for n in lens)
        return {"bytes": tok * c["Hkv"] * (c["d"] + c["d"] // 8) + 4 * c["B"] * c["Hq"] * c["Nq"] * c["d"]
                + 4 * (tok // c["page"]) + 4 * c["B"], "flops": 4 * pairs * c["Hq"] * c["d"]}
    tok = _visible(c["Nk"], c["Nq"], c["window"], c["sinks"])
    pairs = _pairs(c["Nk"] - c["Nq"], c["Nq"], c["window"], c["sinks"])
    return {"bytes": 4 * c["B"] * c["Hkv"] * tok * c["d"] + 4 * c["B"] * c["Hq"] * c["Nq"] * c["d"],
            "flops": 4 * c["B"] * c["Hq"] * pairs * c["d"]}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _exact_attention(q, k, v, pos, tok, W, S):
    """q (Hq, n, d) at positions pos, k and v (Hkv, L, d) of tokens tok, all fp64."""
    Hq, n, d = q.shape
    Hkv = k.shape[0]
    seen = tok[None] <= pos[:, None]
    if W:
        seen &= (tok[None] > pos[:, None] - W) | (tok[None] < S)
    x = torch.einsum("hgnd,hld->hgnl", q.view(Hkv, Hq // Hkv, n, d), k) * d ** -0.5
    x = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
    return torch.einsum("hgnl,hld->hgnd", x, v).reshape(Hq, n, d)


def _exact_quantised(x):
    y = x.double().unflatten(-1, (-1, CHANNELS))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).bfloat16().double()
    n = torch.where(s == 0, torch.zeros_like(y), torch.round((y - lo) / s).clamp(0, 15))
    return (lo + n * s).flatten(-2)


def _exact_record_values(pool, d):
    """Keys and values (pages, Hkv, page, d) in fp64, byte and shift of each channel looked up."""
    dev = pool.device
    t = torch.arange(GROUP, device=dev)[:, None]
    i = torch.arange(d, device=dev)[None]
    kb = t * (d // 2) + (i % 32 // 8) * (d // 8) + (i // 32) * 4 + i % 8 // 2
    ks = (i % 2) * 4 + 0 * t
    vb = (i // 64) * 512 + ((i % 8) * 4 + t % 8 // 2) * 16 + (i % 64 // 16) * 4 + (t % 2) * 2 + t // 8
    vs = (i % 16 // 8) * 4 + 0 * t
    kv, half = [], GROUP * (d // 2 + d // 16)
    for base, byte, shift in ((0, kb, ks), (half, vb, vs)):
        code = ((pool[..., base + byte.flatten()].long() >> shift.flatten()) & 15).double()
        w = pool[..., base + GROUP * d // 2: base + half].long().unflatten(-1, (GROUP, d // 64, 2, 2))
        f = ((w[..., 0] + 256 * w[..., 1]).to(torch.int32) << 16).view(torch.float32).double()
        f = f.repeat_interleave(CHANNELS, -2)            # record's token, channel, (scale, minimum)
        kv.append((code.unflatten(-1, (GROUP, d)) * f[..., 0] + f[..., 1]).flatten(2, 3))
    return kv


def exact(case, seed):
    c = dict(case)
    if c["op"] == "tables":
        return None
    s = prepare(case, seed)
    if c["op"] == "norm_rope":
        rot, ang = c["rot"], s["pos"].double()[:, None, :, None] * s["freq"]
        turn = torch.polar(torch.ones_like(ang), ang)

        def one(x, w):
            y = x.double()
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["d"] + s["eps"])
            y = y if w is None else y * w.double()
            lo, hi = y[..., :rot], y[..., rot:]
            z = lo.unflatten(-1, (-1, 2)) if c["interleaved"] else lo.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            return torch.cat([z, hi], -1)

        return dict(q=one(s["q"], s["wq"]), k=one(s["k"], s["wk"]))
    if c["op"] == "store":
        return dict(k=_exact_quantised(s["k"]), v=_exact_quantised(s["v"]))
    q = s["q"].double()
    out = torch.zeros_like(q)
    if c["op"] == "cache_attn":
        P, W = c["page"], c["window"]
        for b in range(c["B"]):
            n = int(s["lens"][b])
            pages = s["table"][b, : _cdiv(n, P)].long()
            k, v = _exact_record_values(s["pool"][pages], c["d"])
            k, v = (x.transpose(0, 1).flatten(1, 2)[:, :n] for x in (k, v))
            pos = n - c["Nq"] + torch.arange(c["Nq"], device=q.device)
            out[b] = _exact_attention(q[b], k, v, pos, torch.arange(n, device=q.device), W, c["sinks"])
        return out
    Nq, Nk, W, S = c["Nq"], c["Nk"], c["window"], c["sinks"]
    if 4e-12 * c["B"] * c["Hq"] * Nq * min(Nk, W + S + 512) * c["d"] > 8:  # seconds at 1 TFLOP/s of fp64, about
        return None
    for b in range(c["B"]):
        for i in range(0, Nq, 512):
            n = min(512, Nq - i)
            pos = Nk - Nq + i + torch.arange(n, device=q.device)
            lo, hi = max(0, int(pos[0]) - W + 1), int(pos[-1]) + 1
            tok = torch.cat([torch.arange(min(S, lo), device=q.device), torch.arange(lo, hi, device=q.device)])
            out[b, :, i:i + n] = _exact_attention(q[b, :, i:i + n], s["k"][b][:, tok].double(), s["v"][b][:, tok].double(), pos, tok, W, S)
    return out
