"""Where the operators for long shared and multimodal contexts can go wrong: sizes of values, infinities and NaN, places that no call
may read or write, far pools, streams, captured calls that share a workspace.

Tolerances of attention behind a shared prefix (check_prefix).  A bf16 output is off by at most 2^-8 of its value.  P is rounded to f16
and so is each element of the shared V: 2^-11 each of sum P |v|, and beside that at most 2^-15 of the largest scale and 2^-37 of the
largest minimum of the 64 tokens (the documented bound), together below e = 2^-14 max|v|.  Elements of the shared K are off by as much,
so a score by at most (2^-11 + 2^-15) sum |q||k| scale where all tokens' scales are alike, or by sum|q| scale 2^-14 max|k| more
where they are not; that and the exponent's own 2^-20 move the output by at most twice as much times max|v|.  That is the worst case: the roundings
of one row's elements point both ways, so the root mean square of what is off is held to 2^-8 of that of the output (half a bf16
step's, 2^-9 / sqrt 3 of each value, is less than a third of it), except for keys of which many elements are the same number and
round the same way."""
import math

import pytest
import torch

import free_block_sparse_gb300 as fbs
import serving_ref as R
from test_gpu_contexts import bounds_of, check_pages_attn, check_select, i32, loaded, shared
from test_gpu_serving import check_cache_attn, filled, gen, rand, within

pytestmark = pytest.mark.gpu
SHARED = fbs.SPARGE_PREFIX_SHARED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbs.lib()
    yield
    torch.cuda.synchronize()
    assert fbs.device_status() == 0


def check_prefix(q, pool, table, lens, out, d, scale=0.0, even=True, mean=True):
    page, Nq = 16 * pool.shape[2], q.shape[2]
    kn, ks, km, vn, vs, vm = R.read_pool(pool, d)
    K, V = R.dequantise(kn, ks, km), R.dequantise(vn, vs, vm)
    sc = scale or d ** -0.5
    off2 = ref2 = 0.0
    for b, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        k, v = (x[table[b].long()[t // page], :, t % page].transpose(0, 1) for x in (K, V))
        o, a, x = R.attention(q[b].double(), k, v, n - Nq + torch.arange(Nq, device="cuda"), 0, 0, sc, v)
        vmax = torch.nan_to_num(v).abs().amax()
        x = (2.0 ** -11 + 2.0 ** -15) * x
        if not even:
            x = x + q[b].double().abs().sum(-1, keepdim=True) * sc * 2.0 ** -14 * torch.nan_to_num(k).abs().amax()
        within(out[b], o, 2.0 ** -8 * o.abs() + 2.0 ** -10 * a + 2.0 ** -14 * vmax + 2 * (x + 2.0 ** -20) * vmax)
        off2, ref2 = off2 + (out[b].double() - o).square().sum(), ref2 + o.square().sum()
    assert not mean or off2 <= 2.0 ** -16 * ref2


def scaled_tokens(pool, table, b, n, d, page, k_by, v_by, g):
    """Stores n new tokens of sequence b whose keys and values are scaled token by token."""
    H = pool.shape[1]
    t = torch.arange(n, device="cuda")
    k = (rand(g, 1, H, n, d).float() * k_by[None, None, :, None]).bfloat16()
    v = (rand(g, 1, H, n, d).float() * v_by[None, None, :, None]).bfloat16()
    fbs.cache4_store(k, v, (table[b].long()[t // page] * page + t % page)[None].contiguous(), pool)


# ------------------------------------------------------------------------------------------------ shared prefix
@pytest.mark.parametrize("Hq,Hkv,Nq,d,B", [(8, 2, 1, 128, 3), (8, 1, 2, 64, 20), (4, 2, 3, 128, 30), (4, 4, 1, 64, 2)])
@pytest.mark.parametrize("kind", ["climbing", "falling", "tiles", "outliers", "small", "large"])
def test_prefix_values_of_any_size(Hq, Hkv, Nq, d, B, kind):
    g = gen(51)
    page, prefix = 16, 1024
    pool, pages, table, lens = shared(g, prefix, [9 + b for b in range(B)], Hkv, d, page)
    n = prefix
    t = torch.arange(n, device="cuda")
    one = torch.ones(n, device="cuda")
    # V's powers of two differ by 2^18 between tiles while P does not: the unit of the sums follows
    k_by, v_by, even = {
        "climbing": (one, 2.0 ** (-9 + t // 64 % 19), True), "falling": (one, 2.0 ** (9 - t // 64 % 19), True),
        "tiles": (2.0 ** (t // 64 % 3 - 2), 2.0 ** (12 * (t // 64 % 2)), True),
        "outliers": (torch.where(t % 64 == 5, 8 * one, one), torch.where(t % 64 == 9, 1024 * one, one), False),
        "small": (2.0 ** -60 * one, 2.0 ** -90 * one, True), "large": (2.0 ** 30 * one, 2.0 ** 80 * one, True),
    }[kind]
    scaled_tokens(pool, table, 0, n, d, page, k_by, v_by, g)
    if kind in ("small", "large"):  # the sequences' own tokens as well
        for b, m in enumerate(lens):
            s = torch.arange(prefix, m, device="cuda")
            k, v = rand(g, 1, Hkv, m - prefix, d).float() * k_by[0], rand(g, 1, Hkv, m - prefix, d).float() * v_by[0]
            fbs.cache4_store(k.bfloat16(), v.bfloat16(), (table[b].long()[s // page] * page + s % page)[None].contiguous(), pool)
    q = rand(g, B, Hq, Nq, d)
    if kind == "large":
        q = (q.float() * 2.0 ** -30).bfloat16()
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=SHARED)
    check_prefix(q, pool, table, lens, out, d, even=even)


@pytest.mark.parametrize("d,rows", [(128, 3), (128, 60), (64, 3), (64, 60)])
def test_prefix_scores_that_climb_and_peak(d, rows):
    """The reference moves at every tile, or one token late in the prefix takes everything."""
    g = gen(52)
    page, prefix, Hkv, G = 16, 1280, 1, 4
    pool, pages, table, lens = shared(g, prefix, [5 + b for b in range(rows)], Hkv, d, page)
    t = torch.arange(prefix, device="cuda")
    u = torch.sign(torch.randn(d, generator=g, device="cuda"))
    for by in (t / 100.0, (prefix - t) / 100.0, torch.where(t == 1111, 12.0, 0.0)):
        k = (u[None] * by[:, None] + 0.05 * torch.randn(prefix, d, generator=g, device="cuda")).bfloat16()
        v = rand(g, 1, 1, prefix, d)
        fbs.cache4_store(k[None, None].contiguous(), v, (table[0].long()[t // page] * page + t % page)[None].contiguous(), pool)
        q = (u[None, None, None] + 0.1 * torch.randn(rows, G, 1, d, generator=g, device="cuda")).bfloat16()
        q[rows // 2] *= -1
        out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=SHARED)
        check_prefix(q, pool, table, lens, out, d, mean=False)


@pytest.mark.parametrize("B", [3, 60])
def test_prefix_rows_stand_apart(B):
    """A NaN or an infinity in a query row spoils that row alone; zero rows and rows of one value are rows."""
    g = gen(53)
    d, page, prefix, H, G = 128, 16, 640, 2, 3
    pool, pages, table, lens = shared(g, prefix, [7] * B, H, d, page)
    q = rand(g, B, H * G, 1, d)
    q[1, 4] = 0.0
    q[2, 1] = 5e-39
    clean = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=SHARED)
    check_prefix(q, pool, table, lens, clean, d)
    bad = q.clone()
    bad[0, 2, 0, 77], bad[B - 1, 5, 0, 3] = math.nan, math.inf
    out = fbs.cache4_prefix_attn(bad, pool, pages, table, i32(*lens), path=SHARED)
    assert torch.isnan(out[0, 2]).all() and not torch.isfinite(out[B - 1, 5]).any()
    same = torch.ones(B, H * G, dtype=torch.bool, device="cuda")
    same[0, 2] = same[B - 1, 5] = False
    assert torch.equal(out[same], clean[same])


@pytest.mark.parametrize("d", [64, 128])
def test_prefix_tokens_that_are_not_finite(d):
    """A NaN in a shared key spoils its head's rows, one in a value its 64 channels; the tokens beside it keep their values."""
    g = gen(54)
    page, prefix, H, G, B = 16, 640, 2, 2, 3
    pool, pages, table, lens = shared(g, prefix, [7, 30, 1], H, d, page)
    q = rand(g, B, H * G, 1, d)
    clean = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=SHARED)
    # the value's word of token 3 of a record in the middle, last group of 64 channels: a scale that is a NaN
    v_word = 9 * d + 8 * d + (3 * (d // 64) + d // 64 - 1) * 4
    spoilt = pool.clone()
    spoilt[int(pages[20]), 0, 0, v_word:v_word + 2] = 255
    out = fbs.cache4_prefix_attn(q, spoilt, pages, table, i32(*lens), path=SHARED)
    assert torch.isnan(out[:, :G, :, d - 64:]).all()
    assert torch.equal(out[:, :G, :, :d - 64], clean[:, :G, :, :d - 64]) and torch.equal(out[:, G:], clean[:, G:])
    k_word = 8 * d + 3 * (d // 64) * 4
    spoilt = pool.clone()
    spoilt[int(pages[20]), 1, 0, k_word:k_word + 2] = 255
    out = fbs.cache4_prefix_attn(q, spoilt, pages, table, i32(*lens), path=SHARED)
    assert torch.isnan(out[:, G:]).all() and torch.equal(out[:, :G], clean[:, :G])


def test_prefix_path_of_its_own_is_the_cache_attention():
    """Few sequences: bit for bit what the cache attention gives; and the shared path is reproducible, whatever the workspace held."""
    g = gen(55)
    d, page, prefix = 128, 64, 1024
    pool, pages, table, lens = shared(g, prefix, [90, 2, 33], 2, d, page)
    q = rand(g, 3, 8, 2, d)
    kv = i32(*lens)
    assert torch.equal(fbs.cache4_prefix_attn(q, pool, pages, table, kv), fbs.cache4_attn(q, pool, table, kv))
    L = fbs.lib()
    need = L.sparge_cache4_prefix_attn_workspace_bytes(3, 8, 2, 2, d)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        outs.append(fbs.cache4_prefix_attn(q, pool, pages, table, kv, ws=ws, path=SHARED))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check_prefix(q, pool, table, lens, outs[0], d)
    with pytest.raises(fbs.SpargeError):
        fbs.cache4_prefix_attn(q, pool, pages, table, kv, path=2)


def test_prefix_rows_and_pages_that_no_call_touches():
    """Rows behind the batch and pages that no sequence has stay as they were; the pool is only read."""
    g = gen(56)
    d, page, prefix, B = 64, 16, 320, 5
    pool, pages, table, lens = shared(g, prefix, [20] * B, 1, d, page)
    q = rand(g, B, 3, 1, d)
    before = pool.clone()
    wide = torch.full((B + 2, 4, 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[1:B + 1, 1:, 1:2]
    fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), out=out, path=SHARED)
    check_prefix(q, pool, table, lens, out, d)
    assert torch.equal(pool, before)
    wide[1:B + 1, 1:, 1:2] = 7.0
    assert (wide == 7.0).all()


def test_pool_past_32_bits():
    """Pages behind the first 2^32 bytes of a pool and 2^31 of its bounds: every call that takes a pool."""
    d, page, H = 128, 16, 2
    n_pages = 2 ** 22 + 50                                    # 4608 bytes each: 19 GB; bounds of 544: 2.3 GB
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g = gen(57)
    pool = torch.empty(n_pages, H, 1, 18 * d, dtype=torch.uint8, device="cuda")
    bounds = fbs.cache4_bounds(n_pages, H, d)
    need, prefix = 60, 320
    ids = (n_pages - 1 - torch.randperm(need, generator=g, device="cuda")).to(torch.int32)
    table = torch.stack([torch.cat([ids[:20], ids[20:40]]), torch.cat([ids[:20], ids[40:]])]).contiguous()
    lens = [640, 333]
    for b, n in enumerate(lens):
        scaled_tokens(pool, table, b, n, d, page, torch.ones(n, device="cuda"), torch.ones(n, device="cuda"), gen(58 + 0 * b))
    small = pool[n_pages - need:].contiguous()
    near = (table - (n_pages - need)).contiguous()
    kv = i32(*lens)
    q = rand(g, 2, 8, 1, d)
    fbs.cache4_bounds_update(pool, table, kv, 640, bounds)
    b2 = fbs.cache4_bounds(need, H, d)
    fbs.cache4_bounds_update(small, near, kv, 640, b2)
    assert torch.equal(bounds[n_pages - need:], b2)
    got, want = fbs.cache4_select(q, pool, bounds, table, kv, 9), fbs.cache4_select(q, small, b2, near, kv, 9)
    assert torch.equal(torch.where(got[0] >= 0, got[0] - (n_pages - need), got[0]), want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(fbs.cache4_pages_attn(q, pool, *got), fbs.cache4_pages_attn(q, small, *want))
    x = fbs.cache4_prefix_attn(q, pool, ids[:20].contiguous(), table, kv, path=SHARED)
    y = fbs.cache4_prefix_attn(q, small, near[0, :20].contiguous(), near, kv, path=SHARED)
    assert torch.equal(x, y)
    hi = fbs.cache4_bounds_load(pool, bounds, ids[:3].contiguous())[0]
    assert torch.equal(hi, fbs.cache4_bounds_load(small, b2, near[0, :3].contiguous())[0])


# ------------------------------------------------------------------------------------------------ selection, pages
def test_select_many_lists_and_wide_groups():
    """More lists than CTAs, groups of 64 heads, ragged lengths, the same page more than once in a table."""
    g = gen(61)
    d, page = 64, 16
    lens = [1 + (37 * i) % 900 for i in range(40)]
    pool, table = filled(g, lens, 2, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], 2, d)
    kv = i32(*lens)
    fbs.cache4_bounds_update(pool, table, kv, 900, bounds)
    q = rand(g, 40, 4, 3, d)
    check_select(q, pool, table, lens, bounds, 11, 1, 1, fbs.cache4_select(q, pool, bounds, table, kv, 11))
    wide = rand(g, 40, 128, 1, d)
    got = fbs.cache4_select(wide, pool, bounds, table, kv, 7, first=0, last=2)
    check_select(wide, pool, table, lens, bounds, 7, 0, 2, got)
    check_pages_attn(wide[:3], pool, got[0][:3], got[1][:3], fbs.cache4_pages_attn(wide, pool, *got)[:3])
    twice = table.clone()
    long = max(range(40), key=lambda i: lens[i])
    twice[long, 3], twice[long, 9] = table[long, 5], table[long, 5]
    got = fbs.cache4_select(q, pool, bounds, twice, kv, 11)
    check_select(q, pool, twice, lens, bounds, 11, 1, 1, got)
    check_pages_attn(q[long:long + 1], pool, got[0][long:long + 1], got[1][long:long + 1],
                     fbs.cache4_pages_attn(q, pool, *got)[long:long + 1])
    with pytest.raises(fbs.SpargeError):
        fbs.cache4_select(rand(g, 40, 130, 1, d), pool, bounds, table, kv, 7)


def test_select_rows_that_are_not_finite():
    """A query row with a NaN or an infinity has no say: its group's other rows choose; groups without one choose the earliest."""
    g = gen(62)
    d, page, n = 128, 16, 1600
    pool, table = filled(g, [n], 2, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], 2, d)
    kv = i32(n)
    fbs.cache4_bounds_update(pool, table, kv, n, bounds)
    for bad in (math.nan, math.inf, -math.inf):
        q = rand(g, 1, 4, 1, d)
        q[0, 1, 0, 5] = q[0, 2, 0, 90] = q[0, 3, 0, 0] = bad
        check_select(q, pool, table, [n], bounds, 12, 1, 1, fbs.cache4_select(q, pool, bounds, table, kv, 12))
    tiny = rand(g, 1, 4, 1, d).float()
    for by in (2.0 ** -120, 2.0 ** 110):
        q = (tiny * by).bfloat16()
        check_select(q, pool, table, [n], bounds, 12, 1, 1, fbs.cache4_select(q, pool, bounds, table, kv, 12))


def test_select_of_the_longest_tables():
    """32768 columns, a list of all of them but one, and what is refused above."""
    g = gen(63)
    d, page, n_pages = 64, 16, 32768
    pool, table = filled(g, [n_pages * page], 1, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], 1, d)
    kv = i32(n_pages * page)
    fbs.cache4_bounds_update(pool, table, kv, n_pages * page, bounds)
    q = rand(g, 1, 2, 1, d)
    hi, lo = loaded(pool, bounds)
    import contexts_ref as C
    ids = table[0].cpu().long()
    s = C.scores(q[0, :, 0].double(), hi[ids, 0], lo[ids, 0])
    for keep in (100, n_pages - 1):
        pages, lens = fbs.cache4_select(q, pool, bounds, table, kv, keep)
        rest = torch.argsort(s[1:-1], descending=True, stable=True)[:keep - 2] + 1
        want = torch.cat([torch.tensor([0, n_pages - 1]), rest]).sort().values
        assert torch.equal(pages[0, 0, 0].cpu().long(), ids[want])
        assert int(lens[0, 0]) == keep * page
    more = torch.cat([table, table[:, :1]], 1).contiguous()
    with pytest.raises(fbs.SpargeError):
        fbs.cache4_select(q, pool, bounds, more, kv, 100)


def test_pages_lists_of_any_length():
    """Empty lists, lists of one token, lengths above the list's pages, negative ones."""
    g = gen(64)
    d, page = 128, 32
    pool, table = filled(g, [500, 300], 1, d, page)
    q = rand(g, 2, 4, 3, d)
    pages = table[:, None, None, :8].expand(2, 3, 1, 8).contiguous()
    lens = i32(0, 1, 256, 33, 255, 31).view(2, 3)
    out = fbs.cache4_pages_attn(q, pool, pages, lens)
    check_pages_attn(q, pool, pages, lens, out)
    assert (out[0, :, 0] == 0).all()
    odd = fbs.cache4_pages_attn(q, pool, pages, i32(-7, 1, 2 ** 31 - 1, 33, 255, 31).view(2, 3))
    assert torch.equal(odd, out)
    none = fbs.cache4_pages_attn(q, pool, pages[..., :0].contiguous(), lens)
    assert (none == 0).all()


# ------------------------------------------------------------------------------------------------ streams, graphs
def _setting(g, B=6, prefix=512):
    d, page, H = 128, 16, 2
    pool, pages, table, lens = shared(g, prefix, [30 + 11 * b for b in range(B)], H, d, page)
    bounds = fbs.cache4_bounds(pool.shape[0], H, d)
    kv = i32(*lens)
    fbs.cache4_bounds_update(pool, table, kv, max(lens), bounds)
    return pool, pages, table, kv, bounds


def test_calls_on_two_streams_at_once():
    g = gen(65)
    pool, pages, table, kv, bounds = _setting(g)
    qs = [rand(g, 6, 8, 1, 128) for _ in range(2)]

    def calls(q):
        some = fbs.cache4_select(q, pool, bounds, table, kv, 9)
        return (*some, fbs.cache4_pages_attn(q, pool, *some), fbs.cache4_prefix_attn(q, pool, pages, table, kv, path=SHARED))

    want = [calls(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls(qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(x, want[i]))


def test_two_graphs_share_workspaces():
    """Two captured calls over one workspace, replayed in turn with other queries: each gives what an eager call gives."""
    g = gen(66)
    pool, pages, table, kv, bounds = _setting(g)
    L = fbs.lib()
    ws = torch.full((max(L.sparge_cache4_prefix_attn_workspace_bytes(6, 8, 2, 2, 128),
                         L.sparge_cache4_select_workspace_bytes(6, 2, 2, table.shape[1])),), 255, dtype=torch.uint8, device="cuda")
    qs = [rand(g, 6, 8, 1, 128), rand(g, 6, 8, 2, 128)]

    def calls(q):
        some = fbs.cache4_select(q, pool, bounds, table, kv, 9, ws=ws)
        return (*some, fbs.cache4_pages_attn(q, pool, *some), fbs.cache4_prefix_attn(q, pool, pages, table, kv, ws=ws, path=SHARED))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(s):
        for q in qs:
            calls(q)
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                outs.append(calls(q))
            graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(3):
        for q in qs:
            q.copy_(rand(g, *q.shape))
        for graph in graphs + graphs[::-1]:
            graph.replay()
        torch.cuda.synchronize()
        for q, out in zip(qs, outs):
            assert all(torch.equal(a, b) for a, b in zip(out, calls(q)))


def test_calls_refuse_what_they_cannot_take():
    g = gen(67)
    pool, pages, table, kv, bounds = _setting(g)
    q = rand(g, 6, 8, 1, 128)
    some = fbs.cache4_select(q, pool, bounds, table, kv, 9)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    for bad in (lambda: fbs.cache4_prefix_attn(q, pool, pages.long(), table, kv), lambda: fbs.cache4_prefix_attn(q, pool, pages.cpu(), table, kv),
                lambda: fbs.cache4_prefix_attn(q.float(), pool, pages, table, kv), lambda: fbs.cache4_prefix_attn(q[:5], pool, pages, table, kv),
                lambda: fbs.cache4_prefix_attn(q, pool, torch.cat([pages, pages]), table, kv),
                lambda: fbs.cache4_prefix_attn(q, pool, pages, table, kv, ws=ws[1:]), lambda: fbs.cache4_prefix_attn(q, pool, pages, table, kv, ws=ws[:64]),
                lambda: fbs.cache4_prefix_attn(q, pool, pages, table, kv, scale=-1.0),
                lambda: fbs.cache4_pages_attn(q, pool, some[0][:, :, :1], some[1]), lambda: fbs.cache4_pages_attn(q, pool, some[0], some[1].long()),
                lambda: fbs.cache4_select(q, pool, bounds[:3], table, kv, 9), lambda: fbs.cache4_select(q, pool, bounds, table, kv, 1),
                lambda: fbs.cache4_select(q, pool, bounds, table, kv, 9, ws=ws[:64]),
                lambda: fbs.cache4_bounds_update(pool, table, kv, 1, bounds[:, :64]), lambda: fbs.cache4_bounds_load(pool, bounds, pages.long())):
        with pytest.raises((ValueError, TypeError, fbs.SpargeError)):
            bad()
    assert fbs.device_status() == 0


def test_empty_pools_and_batches():
    """A pool without pages has no token: tables that count some are reported, and nothing is read through them."""
    d, page = 128, 16
    pool, bounds = fbs.cache4_pool(0, page, 2, d), fbs.cache4_bounds(0, 2, d)
    q = torch.ones(3, 4, 1, d, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(3, 40, dtype=torch.int32, device="cuda")
    kv = i32(640, 0, 100)
    fbs.cache4_bounds_update(pool, table, kv, 640, bounds)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    pages, lens = fbs.cache4_select(q, pool, bounds, table, kv, 4)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    assert lens.flatten().tolist() == [64, 0, 52] and (pages[1] == -1).all()
    out = fbs.cache4_pages_attn(q, pool, pages, lens)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG and (out == 0).all()
    for path in (0, SHARED):
        out = fbs.cache4_prefix_attn(q, pool, table[0, :20].contiguous(), table, kv, path=path)
        assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG and (out == 0).all()
    g = gen(68)
    pool, pages, table, kv, bounds = _setting(g)
    none = pool.new_empty(0, 8, 1, 128).view(torch.bfloat16).new_empty(0, 8, 1, 128)
    assert fbs.cache4_prefix_attn(none, pool, pages, table[:0], kv[:0], path=SHARED).shape == (0, 8, 1, 128)
    got = fbs.cache4_select(none, pool, bounds, table[:0], kv[:0], 4)
    assert got[0].shape == (0, 1, 2, 4) and fbs.cache4_pages_attn(none, pool, *got).shape == (0, 8, 1, 128)


@pytest.mark.parametrize("Hq,Hkv,Nq,d,own", [(8, 2, 33, 128, [40, 33, 700]), (64, 1, 1, 64, [5, 1, 17]), (64, 1, 3, 128, [5, 100])])
def test_prefix_many_rows_of_a_sequence(Hq, Hkv, Nq, d, own):
    """Chunks of queries and wide groups: rows of one sequence in several row tiles and warps."""
    g = gen(69)
    pool, pages, table, lens = shared(g, 704, own, Hkv, d, 16)
    q = rand(g, len(own), Hq, Nq, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), path=SHARED)
    check_prefix(q, pool, table, lens, out, d)


def test_prefix_lengths_outside_the_table():
    """Negative lengths are nothing, lengths past the table all of it."""
    g = gen(70)
    d, page, prefix = 128, 16, 320
    pool, pages, table, lens = shared(g, prefix, [48, 48, 48], 2, d, page)
    q = rand(g, 3, 4, 2, d)
    want = fbs.cache4_prefix_attn(q, pool, pages, table, i32(368, 0, 368), path=SHARED)
    got = fbs.cache4_prefix_attn(q, pool, pages, table, i32(2 ** 31 - 1, -(2 ** 31), 369), path=SHARED)
    assert torch.equal(want, got) and (got[1] == 0).all()
    check_prefix(q[:1], pool, table[:1], [368], got[:1], d)
