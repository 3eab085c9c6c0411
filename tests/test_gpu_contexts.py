"""The operators for long shared and multimodal contexts on the GPU against their fp64 definitions: rotation over several axes,
page bounds and the selection by them, attention over selected pages, attention behind a shared prefix.

Tolerances.  Rotation and attention over pages as in test_gpu_serving.py (the same arithmetic).  Bounds, selections and lengths are
exact.  Attention behind a prefix rounds the shared keys and values to f16 beside that (test_gpu_contexts_edges.py counts it); the
cases here keep to the cache attention's tolerance all the same, their elements' roundings pointing both ways."""
import math

import pytest
import torch

import contexts_ref as C
import free_block_sparse_gb300 as fbs
import serving_ref as R
from test_gpu_serving import check_cache_attn, filled, gen, rand, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbs.lib()
    assert torch.cuda.is_available()
    yield
    torch.cuda.synchronize()
    assert fbs.device_status() == 0


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------ rotation over several axes
@pytest.mark.parametrize("B,Hq,Hkv,N,d,sections,woven,interleaved,weights,far", [
    (1, 1, 1, 1, 64, (32,), False, False, False, 0),
    (1, 32, 8, 1, 128, (16, 24, 24), False, False, True, 131071),
    (3, 5, 1, 7, 128, (11, 0, 21), True, False, True, 1000),
    (2, 4, 2, 33, 64, (5, 4, 4, 3), True, True, True, 1 << 20),
    (2, 4, 4, 17, 128, (30, 34), False, True, False, (1 << 31) - 4000),
    (1, 3, 2, 5, 64, (1, 7), False, False, True, -70000),
    (1, 2, 2, 9, 128, (), False, False, True, 0),
    (2, 40, 8, 700, 128, (24, 20, 20), True, False, True, 5),
    (1, 17, 3, 2049, 64, (8, 8, 8), False, True, True, 99),
])
def test_axes(B, Hq, Hkv, N, d, sections, woven, interleaved, weights, far):
    g = gen(31)
    q, k = rand(g, B, Hq, N, d, std=3.0), rand(g, B, Hkv, N, d)
    axes = fbs.rope_axes(sections, woven)
    pairs, A = sum(sections), max(1, len(sections))
    assert axes.tolist().count(0) == (sections[0] if sections else 0) and axes.numel() == pairs
    freq = fbs.rope_freqs(2 * pairs, 500000.0)
    pos = (far + torch.randint(0, 3000, (A, B, N), generator=g, device="cuda")).to(torch.int32)
    wq, wk = ((1 + 0.5 * torch.randn(d, generator=g, device="cuda")) if weights else None for _ in range(2))
    a, b = fbs.qk_norm_rope_axes(q, k, freq, axes, pos, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved)
    for x, w, y in ((q, wq, a), (k, wk, b)):
        ref, mag = C.norm_rope_axes(x.double(), w, freq, axes.tolist(), pos, 1e-5, interleaved)
        within(y, ref, 2.0 ** -8 * ref.abs() + (2.0 ** -19 + 2.0 ** -50 * abs(far)) * mag)


def test_axes_of_one_axis_is_the_plain_rotation():
    """The same position on every axis gives bit for bit what the plain call gives."""
    g = gen(32)
    q, k = rand(g, 2, 6, 50, 128), rand(g, 2, 2, 50, 128)
    freq, pos = fbs.rope_freqs(128), torch.randint(0, 1 << 20, (2, 50), generator=g, device="cuda").to(torch.int32)
    want = fbs.qk_norm_rope(q, k, freq, positions=pos)
    for A in (1, 2, 3, 4):
        axes = torch.randint(0, A, (64,), generator=g, device="cuda").to(torch.int32)
        got = fbs.qk_norm_rope_axes(q, k, freq, axes, pos[None].expand(A, -1, -1))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_axes_strides_in_place_and_bad_axes():
    g = gen(33)
    B, Hq, Hkv, N, d = 2, 6, 2, 50, 64
    q = rand(g, B, N, Hq + 1, d)[:, :, :Hq].transpose(1, 2)
    k = rand(g, B, N, Hkv, d).transpose(1, 2)
    freq, axes = fbs.rope_freqs(d), fbs.rope_axes((10, 12, 10))
    wide = torch.randint(0, 5000, (3, 1, N + 7), generator=g, device="cuda").to(torch.int32)
    pos = wide[:, :, 5:5 + N].expand(3, B, N)                       # shared by the batch, rows of a wider array
    a, b = fbs.qk_norm_rope_axes(q, k, freq, axes, pos)
    c, e = fbs.qk_norm_rope_axes(q.contiguous(), k.contiguous(), freq, axes, pos.contiguous())
    assert torch.equal(a, c) and torch.equal(b, e)
    q2, k2 = q.clone(memory_format=torch.preserve_format), k.clone()
    fbs.qk_norm_rope_axes(q2, k2, freq, axes, pos, q_out=q2, k_out=k2)
    assert torch.equal(q2, a) and torch.equal(k2, b)
    bad = axes.clone()
    bad[3], bad[20] = -1, 3
    f0 = freq.clone()
    f0[3] = f0[20] = 0.0                                            # those pairs do not turn
    got = fbs.qk_norm_rope_axes(q, k, freq, bad, pos)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    want = fbs.qk_norm_rope_axes(q, k, f0, axes, pos)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    empty = fbs.qk_norm_rope_axes(q[:, :, :0], k[:, :, :0], freq, axes, pos[:, :, :0])
    assert empty[0].shape == (B, Hq, 0, d)


def test_grid_positions():
    pos = fbs.rope_grid_positions(3, 2, 3, 4)
    assert pos.shape == (3, 1, 27) and pos[:, 0, :3].tolist() == [[0, 1, 2]] * 3
    at = pos[:, 0, 3:].reshape(3, 2, 3, 4) - 3
    for x in range(3):
        n = (2, 3, 4)[x]
        assert torch.equal(at[x].movedim(x, -1), torch.arange(n, device="cuda", dtype=torch.int32).expand(*[m for i, m in enumerate((2, 3, 4)) if i != x], n))
    order = torch.from_numpy(fbs.hilbert_perm_3d(3, 2, 3, 4)).cuda()
    assert torch.equal(fbs.rope_grid_positions(3, 2, 3, 4, order=order), pos[:, :, order.long()])


# ------------------------------------------------------------------------------------------------ bounds
def bounds_of(pool, table, lens, d):
    """hi, lo (pages, H, d) fp64 of the pages of the sequences, by the definition; NaN rows elsewhere."""
    page = 16 * pool.shape[2]
    K = R.dequantise(*R.read_pool(pool, d)[:3])
    hi = torch.full((pool.shape[0], pool.shape[1], d), math.nan, dtype=torch.float64)
    lo = hi.clone()
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            p = int(table[b, j])
            for h in range(pool.shape[1]):
                hi[p, h], lo[p, h], _ = C.page_bounds(K[p, h, :min(page, n - j * page)])
    return hi, lo


def loaded(pool, bounds):
    hi, lo = fbs.cache4_bounds_load(pool, bounds, torch.arange(pool.shape[0], dtype=torch.int32, device="cuda"))
    return hi.double().cpu(), lo.double().cpu()


@pytest.mark.parametrize("H,d,page,lens", [
    (1, 64, 16, [1]), (8, 128, 64, [64, 65, 0, 15, 16, 17, 200]), (3, 128, 16, [100, 3]), (5, 64, 256, [300, 700, 255]),
    (2, 128, 128, [1000]), (4, 64, 32, [33, 31, 32]),
])
def test_bounds(H, d, page, lens):
    g = gen(34)
    pool, table = filled(g, lens, H, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], H, d)
    fbs.cache4_bounds_update(pool, table, i32(*lens), max(lens), bounds)
    got = loaded(pool, bounds)
    want = bounds_of(pool, table, lens, d)
    have = torch.isfinite(want[0])
    for x, y in zip(got, want):
        assert torch.equal(x[have], y[have])
        assert (x[torch.isnan(y)] == 0).all()          # pages that no sequence has
    # no key lies outside, and each bound is within a unit of one
    assert (want[0][have] >= want[1][have]).all()


def test_bounds_of_appended_tokens():
    """N new tokens renew the pages that they lie on, and no other one."""
    g = gen(35)
    lens, d, page, H = [40, 16, 5, 77, 1], 64, 16, 3
    pool, table = filled(g, lens, H, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], H, d)
    bounds.random_(0, 256, generator=g)
    for N in (0, 1, 2, 20):
        before = bounds.clone()
        fbs.cache4_bounds_update(pool, table, i32(*lens), N, bounds)
        want = bounds_of(pool, table, lens, d)
        got = loaded(pool, bounds)
        hit = set()
        for b, n in enumerate(lens):
            for j in range(max(n - N, 0) // page, -(-n // page) if N else 0):
                hit.add(int(table[b, j]))
        for p in range(pool.shape[0]):
            if p in hit:
                assert torch.equal(got[0][p], want[0][p]) and torch.equal(got[1][p], want[1][p])
            else:
                assert torch.equal(bounds[p], before[p])


@pytest.mark.parametrize("d", [64, 128])
def test_bounds_of_values_of_any_size(d):
    """Zeros, equal values, subnormal ones, ones near the largest, an infinity: the unit's two ends."""
    g = gen(36)
    page, n = 16, 16 * 8
    pool = fbs.cache4_pool(8, page, 2, d)
    k = rand(g, 1, 2, n, d)
    k[0, 0, :16] = 0.0
    k[0, 1, :16] = -3.0
    k[0, 0, 16:32] *= 1e-38
    k[0, 1, 16:32] *= 3e37
    k[0, 0, 32:48] = 1.984375                             # 127 * 2^-6: the unit is 2^-6
    k[0, 1, 32:48] = 1.9921875                            # one step further: 2^-5
    k[0, 0, 50, 3] = math.inf
    k[0, 1, 70, 5] = math.nan
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    fbs.cache4_store(k, k, torch.arange(n, device="cuda")[None], pool)
    bounds = fbs.cache4_bounds(8, 2, d)
    fbs.cache4_bounds_update(pool, table, i32(n), n, bounds)
    got, want = loaded(pool, bounds), bounds_of(pool, table, [n], d)
    # (products and sums of the codes are fp32 in the call: values near 1e-38 may round there)
    for x, y in zip(got, want):
        assert torch.equal(x, y) or ((x - y).abs() <= 2.0 ** -126)[torch.isfinite(y)].all()
    assert torch.isinf(got[0][3, 0]).all() and torch.isinf(got[1][4, 1]).all()
    assert torch.isfinite(got[0][3, 1]).all() and torch.isfinite(got[0][4, 0]).all()


def test_bounds_bad_pages_and_lengths():
    g = gen(37)
    d, page, H = 128, 16, 2
    pool, table = filled(g, [64, 64], H, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], H, d)
    bad = table.clone()
    bad[0, 1], bad[1, 2] = -1, pool.shape[0]
    fbs.cache4_bounds_update(pool, bad, i32(64, 64), 64, bounds)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    assert (bounds[int(table[0, 1])] == 0).all() and (bounds[int(table[1, 2])] == 0).all() and (bounds[int(table[0, 0])] != 0).any()
    one, two = bounds.clone().zero_(), bounds.clone().zero_()
    fbs.cache4_bounds_update(pool, table, i32(2 ** 31 - 1, -5), 2 ** 40, one)
    fbs.cache4_bounds_update(pool, table, i32(64, 0), 64, two)
    assert torch.equal(one, two)
    hi, lo = fbs.cache4_bounds_load(pool, one, i32(-1, pool.shape[0], int(table[0, 0])))
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    assert (hi[:2] == 0).all() and (lo[:2] == 0).all() and (hi[2] != 0).any()
    assert fbs.cache4_bounds_load(pool, one, i32())[0].shape == (0, H, d)


# ------------------------------------------------------------------------------------------------ selection
def check_select(q, pool, table, lens, bounds, keep, first, last, got):
    page, d = 16 * pool.shape[2], q.shape[3]
    B, Hq, Nq = q.shape[:3]
    H = pool.shape[1]
    hi, lo = loaded(pool, bounds)
    pages, out_lens = got[0].cpu(), got[1].cpu()
    tab, qq = table.cpu(), q.double()
    for b in range(B):
        for i in range(Nq):
            seen = max(0, min(lens[b], table.shape[1] * page) - Nq + 1 + i)
            n = -(-seen // page)
            m = min(n, keep)
            assert int(out_lens[b, i]) == ((m - 1) * page + (seen - 1) % page + 1 if m else 0)
            ids = tab[b, :n].long()
            for h in range(H):
                G = Hq // H
                s = C.scores(qq[b, h * G:(h + 1) * G, i], hi[ids, h], lo[ids, h])
                want = [int(ids[j]) for j in C.choose(s.tolist(), keep, first, last)]
                assert pages[b, i, h].tolist() == want + [-1] * (keep - m), (b, i, h)


@pytest.mark.parametrize("Hq,Hkv,Nq,d,page,lens,keep,first,last", [
    (1, 1, 1, 64, 16, [1], 1, 0, 1),
    (4, 1, 1, 128, 64, [1, 0, 64, 65, 700], 4, 1, 1),
    (32, 8, 1, 128, 16, [2000, 15, 333], 20, 1, 2),
    (8, 8, 1, 64, 32, [300, 5, 1000], 1000, 3, 5),      # everything fits
    (6, 2, 5, 64, 16, [2, 5, 700], 7, 1, 1),            # a sequence shorter than its queries
    (16, 1, 3, 128, 16, [500, 33], 3, 1, 2),            # nothing left to choose
    (64, 1, 1, 64, 16, [900], 12, 0, 1),                # the most heads of a group
    (10, 2, 7, 128, 16, [900, 6], 9, 2, 3),
    (3, 3, 1, 64, 16, [20000], 100, 1, 1),              # a cluster of CTAs per list
    (4, 2, 2, 128, 16, [40000, 17], 300, 1, 1),
])
def test_select_and_attend(Hq, Hkv, Nq, d, page, lens, keep, first, last):
    g = gen(38)
    pool, table = filled(g, lens, Hkv, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], Hkv, d)
    kv = i32(*lens)
    fbs.cache4_bounds_update(pool, table, kv, max(lens), bounds)
    q = rand(g, len(lens), Hq, Nq, d)
    q[0, 0, 0] = 0.0
    got = fbs.cache4_select(q, pool, bounds, table, kv, keep, first=first, last=last)
    check_select(q, pool, table, lens, bounds, keep, first, last, got)
    out = fbs.cache4_pages_attn(q, pool, *got)
    check_pages_attn(q, pool, got[0], got[1], out)


def check_pages_attn(q, pool, pages, lens, out, scale=0.0):
    B, Hq, Nq, d = q.shape
    H, G = pool.shape[1], q.shape[1] // pool.shape[1]
    for b in range(B):
        for i in range(Nq):
            for h in range(H):
                check_cache_attn(q[b:b + 1, h * G:(h + 1) * G, i:i + 1], pool[:, h:h + 1], pages[b, i, h][None], [int(lens[b, i])],
                                 out[b:b + 1, h * G:(h + 1) * G, i:i + 1], d, scale=scale)


@pytest.mark.parametrize("d,page,n_pages", [(64, 16, 3000), (128, 16, 700), (128, 64, 257)])
def test_select_of_equal_scores(d, page, n_pages):
    """Equal scores go to the earliest pages: pages that all hold the same keys, a few better ones among them."""
    pool = fbs.cache4_pool(n_pages, page, 1, d)
    k = torch.ones(1, 1, n_pages * page, d, device="cuda", dtype=torch.bfloat16)
    better = [n_pages - 2, 5, n_pages // 2]
    for p in better:
        k[0, 0, p * page] = 2.0
    fbs.cache4_store(k, k, torch.arange(n_pages * page, device="cuda")[None], pool)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    bounds = fbs.cache4_bounds(n_pages, 1, d)
    n = n_pages * page
    fbs.cache4_bounds_update(pool, table, i32(n), n, bounds)
    q = torch.ones(1, 2, 1, d, device="cuda", dtype=torch.bfloat16)
    pages, lens = fbs.cache4_select(q, pool, bounds, table, i32(n), 10, first=0, last=1)
    assert pages[0, 0, 0].tolist() == sorted([0, 1, 2, 3, 4, 6] + better + [n_pages - 1])
    pages, _ = fbs.cache4_select(-q, pool, bounds, table, i32(n), 4, first=1, last=1)   # the better ones are no worse for -q: lo is 1
    assert pages[0, 0, 0].tolist() == [0, 1, 2, n_pages - 1]
    pages, _ = fbs.cache4_select(q * math.nan, pool, bounds, table, i32(n), 4, first=0, last=1)
    assert pages[0, 0, 0].tolist() == [0, 1, 2, n_pages - 1]


def test_select_bounds_hold():
    """A page that is left out holds no key whose product with the rounded query is above the kept pages' scores' smallest, and a
    planted key is found."""
    g = gen(39)
    d, page, n_pages = 128, 16, 400
    pool, table = filled(g, [n_pages * page], 1, d, page)
    u = rand(g, 1, 1, 1, d, std=3.0)
    at = torch.tensor([page * 201 + 7], device="cuda")
    fbs.cache4_store(u, u, (table[0].long()[at // page] * page + at % page)[None].contiguous(), pool)
    bounds = fbs.cache4_bounds(pool.shape[0], 1, d)
    kv = i32(n_pages * page)
    fbs.cache4_bounds_update(pool, table, kv, n_pages * page, bounds)
    pages, _ = fbs.cache4_select(u, pool, bounds, table, kv, 12)
    assert int(table[0, 201]) in pages[0, 0, 0].tolist()
    K = R.dequantise(*R.read_pool(pool, d)[:3])[:, 0]
    hi, lo = loaded(pool, bounds)
    t = C.unit(float(u.double().abs().max()))
    r = t * torch.round(u.double()[0, 0, 0] / t)
    ids = table[0].long()
    best = (K[ids] @ r).amax(-1).cpu()
    assert (best <= C.scores(u[0, 0].double(), hi[ids.cpu(), 0], lo[ids.cpu(), 0])).all()


def test_pages_with_infinities_are_kept():
    g = gen(40)
    d, page, n = 64, 16, 16 * 50
    pool, table = filled(g, [n], 2, d, page)
    inf = torch.full((1, 2, 1, d), 1.0, dtype=torch.bfloat16, device="cuda")
    inf[0, 1, 0, 3] = math.inf
    at = torch.tensor([16 * 31 + 2], device="cuda")
    fbs.cache4_store(inf, inf, (table[0].long()[at // page] * page + at % page)[None].contiguous(), pool)
    bounds = fbs.cache4_bounds(pool.shape[0], 2, d)
    fbs.cache4_bounds_update(pool, table, i32(n), n, bounds)
    q = rand(g, 1, 2, 1, d)
    pages, lens = fbs.cache4_select(q, pool, bounds, table, i32(n), 3)
    assert int(table[0, 31]) == int(pages[0, 0, 1, 1])
    out = fbs.cache4_pages_attn(q, pool, pages, lens)
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all()


def test_select_strides_bad_pages_and_given_outputs():
    g = gen(41)
    d, page, lens = 128, 16, [700, 450]
    pool, table = filled(g, lens, 2, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], 2, d)
    kv = i32(*lens)
    fbs.cache4_bounds_update(pool, table, kv, 700, bounds)
    q = rand(g, 2, 3, 7, d).transpose(1, 2)[:, :6]                   # (B, H, N, d) of (B, N, H, d), padded
    wide = torch.full((2, table.shape[1] + 5), 77777, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    pages = torch.empty(2, 3, 2, 9, dtype=torch.int32, device="cuda")
    olens = torch.empty(2, 3, dtype=torch.int32, device="cuda")
    got = fbs.cache4_select(q, pool, bounds, wide[:, :table.shape[1]], kv, 9, pages=pages, lens=olens)
    assert got[0] is pages and got[1] is olens
    check_select(q, pool, table, lens, bounds, 9, 1, 1, got)
    out = torch.empty(2, 3, 6, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    assert fbs.cache4_pages_attn(q, pool, pages, olens, scale=0.3, out=out) is out
    check_pages_attn(q, pool, pages, olens, out, scale=0.3)
    bad = table.clone()
    bad[0, 11], bad[0, 20] = -7, pool.shape[0]
    p2, l2 = fbs.cache4_select(q, pool, bounds, bad, kv, 9)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    assert torch.equal(p2[1], pages[1]) and (p2[0] >= 0).all() and (p2[0] < pool.shape[0]).all()
    # such a page is left out of the attention, and the rest of the list is attended
    spoilt, want = pages.clone(), pages.clone()
    spoilt[0, 0, 0, 3] = pool.shape[0]
    got = fbs.cache4_pages_attn(q, pool, spoilt, olens)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    good = fbs.cache4_pages_attn(q, pool, want, olens)
    assert torch.equal(got[1], good[1]) and torch.equal(got[0, :, 1:], good[0, :, 1:]) and torch.isfinite(got.float()).all()
    assert fbs.cache4_pages_attn(q[:0], pool, pages[:0], olens[:0]).shape == (0, 6, 3, d)


# ------------------------------------------------------------------------------------------------ shared prefix
def shared(g, prefix, own, H, d, page, std=1.0):
    """A pool whose sequences share `prefix` tokens and have own[b] of their own; prefix pages, tables, lengths."""
    np_ = prefix // page
    need = [-(-n // page) for n in own]
    ids = torch.randperm(np_ + sum(need) + 3, generator=g, device="cuda").to(torch.int32)
    pool = fbs.cache4_pool(np_ + sum(need) + 3, page, H, d)
    pool.fill_(255)
    table = torch.full((len(own), np_ + max(need + [1])), -1, dtype=torch.int32, device="cuda")
    table[:, :np_] = ids[:np_]
    at = np_
    stretches = [(ids[:np_], prefix)]
    for b, n in enumerate(own):
        table[b, np_:np_ + need[b]] = ids[at:at + need[b]]
        stretches.append((ids[at:at + need[b]], n))
        at += need[b]
    for pages, n in stretches:
        for t0 in range(0, n, 8192):
            m = min(8192, n - t0)
            k, v = rand(g, 1, H, m, d, std=std), rand(g, 1, H, m, d)
            k[..., 3] += 4.0
            v[:, :, m // 2:] *= 30.0
            t = t0 + torch.arange(m, device="cuda")
            fbs.cache4_store(k, v, (pages.long()[t // page] * page + t % page)[None].contiguous(), pool)
    return pool, ids[:np_].contiguous(), table, [prefix + n for n in own]


@pytest.mark.parametrize("Hq,Hkv,Nq,d,page,prefix,own", [
    (1, 1, 1, 64, 16, 16, [1]),
    (4, 1, 1, 128, 64, 64, [1, 64, 65, 15, 16, 17]),
    (8, 2, 1, 128, 64, 1024, [100, 3, 70]),
    (32, 8, 1, 128, 64, 4096, [33] * 5),
    (8, 8, 1, 64, 32, 320, [300, 5, 1000]),
    (6, 2, 5, 64, 16, 48, [5, 700, 6]),                 # a prefix of three records
    (10, 2, 7, 128, 256, 512, [900, 7]),
    (16, 1, 1, 128, 16, 2000, [20 + 3 * i for i in range(30)]),   # 480 rows
    (4, 4, 1, 64, 16, 1008, [1 + i for i in range(140)]),
    (3, 1, 2, 64, 128, 128, [2] * 50),
    (5, 1, 1, 128, 16, 8208, [9]),
])
def test_prefix_attn(Hq, Hkv, Nq, d, page, prefix, own):
    g = gen(42)
    pool, pages, table, lens = shared(g, prefix, own, Hkv, d, page)
    q = rand(g, len(own), Hq, Nq, d)
    q[0, 0, 0] = 0.0
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=fbs.SPARGE_PREFIX_SHARED)
    check_cache_attn(q, pool, table, lens, out, d)


def test_prefix_attn_sequences_that_do_not_hold_it():
    """Padding rows, sequences inside the prefix or with queries in it: any length is taken."""
    g = gen(43)
    d, page, prefix = 128, 16, 320
    pool, pages, table, lens = shared(g, prefix, [40, 3, 4, 1, 0, 9], 2, d, page)
    lens = [lens[0], 323, 324, 321, 0, 150]
    table[4] = -1
    q = rand(g, 6, 4, 4, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=fbs.SPARGE_PREFIX_SHARED)
    check_cache_attn(q, pool, table, lens, out, d)
    assert (out[4] == 0).all()
    none = fbs.cache4_prefix_attn(q, pool, pages[:0], table, i32(*lens), path=fbs.SPARGE_PREFIX_SHARED)
    check_cache_attn(q, pool, table, lens, none, d)
    assert fbs.device_status() == 0


def test_prefix_attn_strides_scale_and_bad_pages():
    g = gen(44)
    d, page, prefix = 64, 16, 640
    pool, pages, table, lens = shared(g, prefix, [50, 10], 2, d, page, std=4.0)
    q = rand(g, 2, 3, 9, d, std=4.0).transpose(1, 2)[:, :8]
    out = torch.empty(2, 3, 8, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    wide = torch.full((2, table.shape[1] + 5), 77777, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert fbs.cache4_prefix_attn(q, pool, pages, wide[:, :table.shape[1]], i32(*lens), scale=0.3, out=out, path=1) is out
    check_cache_attn(q, pool, table, lens, out, d, scale=0.3)
    bad, bad_table = pages.clone(), table.clone()
    bad[1], bad[7], bad[39] = -1, pool.shape[0], 2 ** 31 - 1
    for j in (1, 7, 39):
        bad_table[:, j] = -1
    got = fbs.cache4_prefix_attn(q, pool, bad, bad_table, i32(*lens), path=fbs.SPARGE_PREFIX_SHARED)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    # as if the tokens of those pages were not there
    keep = [j for j in range(table.shape[1]) if j not in (1, 7, 39)]
    check_cache_attn(q, pool, table[:, keep].contiguous(), [n - 48 for n in lens], got, d)
    assert fbs.device_status() == 0


# ------------------------------------------------------------------------------------------------ together
def test_a_step_of_all_of_them():
    """A decoding step as a model's layer makes it: rotation over axes, store, bounds, selection, attention over the selected pages
    and behind the shared prefix, and the same captured into a graph and replayed on other values."""
    g = gen(45)
    B, Hq, Hkv, d, page, prefix = 3, 8, 2, 128, 16, 512
    own = [90, 33, 200]
    pool, pages, table, lens = shared(g, prefix, [n + 1 for n in own], Hkv, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], Hkv, d)
    fbs.cache4_bounds_update(pool, table, i32(*[n - 1 for n in lens]), max(lens), bounds)
    kv = i32(*lens)
    at = kv.long()[:, None] - 1
    slots = torch.gather(table.long(), 1, at // page) * page + at % page
    freq, axes = fbs.rope_freqs(d), fbs.rope_axes((16, 24, 24), woven=True)
    q, k, v = rand(g, B, Hq, 1, d), rand(g, B, Hkv, 1, d), rand(g, B, Hkv, 1, d)
    pos = torch.randint(0, 900, (3, B, 1), generator=g, device="cuda").to(torch.int32)

    def step():
        a, b = fbs.qk_norm_rope_axes(q, k, freq, axes, pos)
        fbs.cache4_store(b, v, slots, pool)
        fbs.cache4_bounds_update(pool, table, kv, 1, bounds)
        some, n = fbs.cache4_select(a, pool, bounds, table, kv, 12, first=2, last=2)
        return a, some, n, fbs.cache4_pages_attn(a, pool, some, n), fbs.cache4_prefix_attn(a, pool, pages, table, kv, path=1)

    def check(a, some, n, near, whole):
        want, mag = C.norm_rope_axes(q.double(), None, freq, axes.tolist(), pos, 1e-6, False)
        within(a, want, 2.0 ** -8 * want.abs() + 2.0 ** -19 * mag)
        check_select(a, pool, table, lens, bounds, 12, 2, 2, (some, n))
        check_pages_attn(a, pool, some, n, near)
        check_cache_attn(a, pool, table, lens, whole, d)
        hi, lo = loaded(pool, bounds)
        w = bounds_of(pool, table, lens, d)
        have = ~torch.isnan(w[0])
        assert torch.equal(hi[have], w[0][have]) and torch.equal(lo[have], w[1][have])

    check(*step())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    for seed in (46, 47):
        g2 = gen(seed)
        q.copy_(rand(g2, B, Hq, 1, d, std=2.0))
        k.copy_(rand(g2, B, Hkv, 1, d))
        v.copy_(rand(g2, B, Hkv, 1, d, std=5.0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(*got)
    assert fbs.device_status() == 0
