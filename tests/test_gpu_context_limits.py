"""Page bounds, selection and attention behind a prefix at their ends, against the fp64 definitions in contexts_ref.py."""
import math

import pytest
import torch

import contexts_ref as C
import free_block_sparse_gb300 as fbs
import serving_ref as R
from test_gpu_contexts import check_select, i32, loaded
from test_gpu_serving import filled, gen, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbs.lib()
    yield
    torch.cuda.synchronize()
    assert fbs.device_status() == 0


# ------------------------------------------------------------------------------------------------ selection
def of_size(g, n, H, d, page, size):
    """A sequence of n tokens whose keys have about this size, and bounds."""
    pool, table = filled(g, [n], H, d, page)
    t = torch.arange(n, device="cuda")
    k = (torch.randn(1, H, n, d, generator=g, device="cuda").double() * size).bfloat16()
    fbs.cache4_store(k, k, (table[0].long()[t // page] * page + t % page)[None].contiguous(), pool)
    bounds = fbs.cache4_bounds(pool.shape[0], H, d)
    fbs.cache4_bounds_update(pool, table, i32(n), n, bounds)
    return pool, table, bounds


@pytest.mark.parametrize("G,Nq,d", [(1, 1, 64), (2, 3, 128), (3, 1, 64), (4, 2, 128), (7, 1, 128), (20, 2, 64)])
@pytest.mark.parametrize("keys,queries", [(100, 30), (110, 110), (-100, -50), (-110, -110), (-60, 60), (115, -20)])
def test_select_scores_of_any_size(G, Nq, d, keys, queries):
    """Products of keys and queries far outside fp32's range rank as they do in 64 bits: heads of a group have sizes 2^5 apart."""
    g = gen(91)
    n, page, H = 1600, 16, 2
    pool, table, bounds = of_size(g, n, H, d, page, 2.0 ** keys)
    q = rand(g, 1, H * G, Nq, d).double() * 2.0 ** queries
    q = (q * 2.0 ** (-5.0 * (torch.arange(H * G, device="cuda") % G % 3))[None, :, None, None]).bfloat16()
    got = fbs.cache4_select(q, pool, bounds, table, i32(n), 12)
    check_select(q, pool, table, [n], bounds, 12, 1, 1, got)


def test_select_large_negative_scores_and_pages_that_are_not_there():
    """Pages with scores of -2^140 are pages: they come in front of places without one."""
    g = gen(92)
    d, page, n = 64, 16, 16 * 60
    pool, table = filled(g, [n], 1, d, page)
    t = torch.arange(n, device="cuda")
    k = (2.0 ** 100 * (1 + torch.rand(1, 1, n, d, generator=g, device="cuda"))).bfloat16()
    fbs.cache4_store(k, k, (table[0].long()[t // page] * page + t % page)[None].contiguous(), pool)
    bounds = fbs.cache4_bounds(pool.shape[0], 1, d)
    fbs.cache4_bounds_update(pool, table, i32(n), n, bounds)
    q = torch.full((1, 2, 1, d), -(2.0 ** 40), dtype=torch.bfloat16, device="cuda")
    bad = table.clone()
    bad[0, 5:25] = -1
    pages, lens = fbs.cache4_select(q, pool, bounds, bad, i32(n), 40)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    there = [j for j in range(60) if not 5 <= j < 25]
    assert pages[0, 0, 0].tolist() == [int(table[0, j]) for j in there] and int(lens[0, 0]) == 40 * page


# ------------------------------------------------------------------------------------------------ bounds
@pytest.mark.parametrize("d,page,H", [(128, 64, 8), (64, 16, 3), (64, 256, 1)])
@pytest.mark.parametrize("B", [2, 7, 300])
def test_bounds_of_a_page_that_sequences_hold_to_different_lengths(B, d, page, H):
    """Forks of one sequence whose last page they share, each up to a token of its own: the page's bounds cover the most of them,
    whatever the order, and one call's are another's."""
    g = gen(93)
    n = 3 * page
    pool, one = filled(g, [n], H, d, page)
    table = one.expand(B, -1).contiguous()
    K = R.dequantise(*R.read_pool(pool, d)[:3])
    for most in (1, 5, page - 1, page):
        lens = 2 * page + 1 + torch.randint(0, most, (B,), generator=g, device="cuda").to(torch.int32)
        lens[int(torch.randint(0, B, (1,), generator=g, device="cuda"))] = 2 * page + most
        for _ in range(20):
            bounds = fbs.cache4_bounds(pool.shape[0], H, d)
            fbs.cache4_bounds_update(pool, table, lens, 1, bounds)
            hi, lo = loaded(pool, bounds)
            p = int(one[0, 2])
            for h in range(H):
                want = C.page_bounds(K[p, h, :most])
                assert torch.equal(hi[p, h], want[0].cpu()) and torch.equal(lo[p, h], want[1].cpu())


def test_bounds_of_a_page_that_a_longer_sequence_has_whole():
    """A sequence that ends on a page which another one has filled leaves the bounds of the whole page as they are."""
    g = gen(94)
    d, page, H = 64, 32, 2
    pool, one = filled(g, [4 * page], H, d, page)
    table, bounds = one.expand(3, -1).contiguous(), fbs.cache4_bounds(pool.shape[0], H, d)
    fbs.cache4_bounds_update(pool, table[:1], i32(4 * page), 4 * page, bounds)
    whole = bounds.clone()
    fbs.cache4_bounds_update(pool, table, i32(page + 3, 4 * page, 7), 1, bounds)
    assert torch.equal(bounds, whole)


@pytest.mark.parametrize("H,d,page,lens", [(8, 128, 64, [64, 65, 0, 15, 200]), (3, 128, 16, [100, 3]), (2, 64, 256, [300, 700])])
def test_bounds_hold_every_key(H, d, page, lens):
    """As loaded, no key of a page lies outside, and each bound is less than a unit from one."""
    g = gen(95)
    pool, table = filled(g, lens, H, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], H, d)
    fbs.cache4_bounds_update(pool, table, i32(*lens), max(lens), bounds)
    hi, lo = loaded(pool, bounds)
    K = R.dequantise(*R.read_pool(pool, d)[:3]).cpu()
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            p = int(table[b, j])
            k = K[p, :, :min(page, n - j * page)]
            assert (k <= hi[p][:, None]).all() and (k >= lo[p][:, None]).all()
            for h in range(H):
                s = C.unit(float(k[h].abs().max()))
                assert (hi[p, h] - k[h].amax(0) < s).all() and (k[h].amin(0) - lo[p, h] < s).all()


@pytest.mark.parametrize("G,d,page,outliers", [(1, 128, 64, False), (4, 128, 64, False), (4, 64, 16, False), (1, 128, 64, True), (4, 64, 16, True)])
def test_selection_beside_unrounded_bounds(G, d, page, outliers):
    """How far the rounding of bounds and queries can move a selection.  A score is at least the row's bound of t r over the page's own
    largest and smallest keys and at most s t sum |r| above it, and a query is off by t / 2 a channel: so no page that is left out has a bound
    (of unrounded keys and queries) above a kept one's by more than s t sum |r| of the kept page and t / 2 sum max|k| of both.  Outliers: one
    key of one in eight pages, in a channel where the queries are zero, doubles that page's unit several times."""
    g = gen(96)
    n_pages, H, keep = 300, 2, 40
    n = n_pages * page
    pool, table = filled(g, [n], H, d, page)
    t = torch.arange(n, device="cuda")
    k = torch.randn(1, H, n, d, generator=g, device="cuda")
    k += 0.5 * torch.randn(1, H, n_pages, 1, d, generator=g, device="cuda").expand(-1, -1, -1, page, -1).reshape(1, H, n, d)
    if outliers:
        k[:, :, ::8 * page, 5] = 40.0
    q = rand(g, 1, H * G, 1, d)
    if outliers:
        q[..., 5] = 0.0
    fbs.cache4_store(k.bfloat16(), k.bfloat16(), (table[0].long()[t // page] * page + t % page)[None].contiguous(), pool)
    bounds = fbs.cache4_bounds(pool.shape[0], H, d)
    fbs.cache4_bounds_update(pool, table, i32(n), n, bounds)
    pages, _ = fbs.cache4_select(q, pool, bounds, table, i32(n), keep)
    K = R.dequantise(*R.read_pool(pool, d)[:3])[table[0].long()].cpu()                # pages, H, tokens, d
    qd = q.double().cpu()[0, :, 0]
    where = {int(p): j for j, p in enumerate(table[0].tolist())}
    for h in range(H):
        hi, lo = K[:, h].amax(1), K[:, h].amin(1)
        s = torch.tensor([C.unit(float(x)) for x in K[:, h].abs().amax((1, 2))], dtype=torch.float64)
        rows = qd[h * G:(h + 1) * G]
        u = torch.maximum(rows[:, None] * hi, rows[:, None] * lo).sum(-1).amax(0)     # the unrounded bound of each page
        ts = [C.unit(float(r.abs().max())) for r in rows]
        off = max(ts) / 2 * torch.maximum(hi.abs(), lo.abs()).sum(-1)
        up = max(float((torch.round(r / x) * x).abs().sum()) for r, x in zip(rows, ts))
        kept = [where[p] for p in pages[0, 0, h].tolist()]
        kept = [j for j in kept if 0 < j < n_pages - 1]
        left = [j for j in range(1, n_pages - 1) if j not in kept]
        assert len(kept) == keep - 2
        assert float((u - off)[left].max()) <= float((u + off + s * up)[kept].min())


# ------------------------------------------------------------------------------------------------ shared prefix
def test_auto_shares_where_that_is_faster():
    """The call that names no path, at a size where sharing takes less time: bit for bit the shared path, which rounds otherwise than
    each sequence by itself."""
    from test_gpu_contexts import shared
    g = gen(97)
    d, page, B = 128, 64, 32
    pool, pages, table, lens = shared(g, 16384, [20 + b for b in range(B)], 2, d, page)
    q = rand(g, B, 8, 1, d)
    auto = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens))
    assert torch.equal(auto, fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=fbs.SPARGE_PREFIX_SHARED))
    assert not torch.equal(auto, fbs.cache4_attn(q, pool, table, i32(*lens)))


@pytest.mark.parametrize("B,Hq,Hkv,Nq,d,prefix,page", [
    (2000, 8, 4, 1, 64, 64, 16),        # 64 items of one tile: several to a CTA, two tiles of rows each
    (300, 64, 64, 1, 128, 80, 16),      # 128 items of two tiles, the second of one record
    (2, 400, 200, 1, 128, 48, 16),      # 200 items of a part of a tile, one tile of rows: the second stream has none
    (3, 120, 60, 2, 64, 208, 16),       # 60 items of four tiles, cut in odd places
])
def test_prefix_of_many_items(B, Hq, Hkv, Nq, d, prefix, page):
    """More items than CTAs, or nearly: pieces of one tile, several for a CTA; a few sequences of all are looked at."""
    from test_gpu_contexts import shared
    from test_gpu_contexts_edges import check_prefix
    g = gen(98)
    pool, pages, table, lens = shared(g, prefix, [Nq + b % 7 for b in range(B)], Hkv, d, page)
    q = rand(g, B, Hq, Nq, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=fbs.SPARGE_PREFIX_SHARED)
    some = torch.tensor(sorted({0, 1, B // 3, B // 2, B - 1}), device="cuda")
    check_prefix(q[some], pool, table[some], [lens[b] for b in some.tolist()], out[some], d)
    assert torch.equal(out, fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=fbs.SPARGE_PREFIX_SHARED))


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_over_the_queries(d):
    """The output in the queries' place gives what one of its own gives: a row's queries are read before it is written."""
    from test_gpu_contexts import shared
    g = gen(99)
    B, page = 40, 16
    pool, pages, table, lens = shared(g, 640, [3 + 5 * b for b in range(B)], 2, d, page)
    kv, bounds = i32(*lens), fbs.cache4_bounds(pool.shape[0], 2, d)
    fbs.cache4_bounds_update(pool, table, kv, max(lens), bounds)
    q = rand(g, B, 8, 3, d)
    some = fbs.cache4_select(q, pool, bounds, table, kv, 20)
    for call in (lambda x, out: fbs.cache4_attn(x, pool, table, kv, out=out),
                 lambda x, out: fbs.cache4_pages_attn(x, pool, *some, out=out),
                 lambda x, out: fbs.cache4_prefix_attn(x, pool, pages, table, kv, out=out, path=fbs.SPARGE_PREFIX_SHARED)):
        x = q.clone()
        assert torch.equal(call(x, x), call(q, None))
