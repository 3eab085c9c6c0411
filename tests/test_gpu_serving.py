"""The serving operators on the GPU against their fp64 definitions: norm and rotation, cache tables, the 4-bit
cache's store and load, the attention over it, and the window attention.

Tolerances.  A bf16 output is off by at most half a step, 2^-8 of its value.  Norm and rotation: about 30
fp32 operations (2^-24 each) on what is summed, 2^-19 of it.  Attention: P rounded to f16 (2^-11) or, with
few rows, to two bf16 (2^-16), times sum P |v| (for the 4-bit cache |scale code|, what P multiplies); scores are
fp32 sums of d <= 128 products, off by at most 2^-16 of sum |q||k| scale, and with the exponent's own error (2^-20)
move the output by at most twice that times the largest |v|."""
import math

import pytest
import torch

import free_block_sparse_gb300 as fbs
import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbs.lib()
    assert torch.cuda.is_available()
    yield
    torch.cuda.synchronize()
    assert fbs.device_status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=g, device="cuda")).bfloat16()


def within(got, ref, tol):
    got = got.double()
    off = (got - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (int(bad.sum()), float((off - tol).max()), float(off.max()))


# ------------------------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot,interleaved,weights,far", [
    (1, 1, 1, 1, 64, 64, False, False, 0),
    (1, 32, 8, 1, 128, 128, False, True, 131071),
    (3, 5, 1, 7, 128, 64, False, True, 1000),
    (2, 4, 2, 33, 64, 32, True, True, 1 << 20),
    (2, 4, 4, 17, 128, 128, True, False, (1 << 31) - 40),
    (1, 3, 2, 5, 64, 16, False, True, -70000),
    (1, 2, 2, 9, 128, 0, False, True, 0),
    (2, 40, 8, 700, 128, 128, False, True, 5),        # several heads per CTA
    (1, 17, 3, 2049, 64, 48, True, True, 99),
])
def test_norm_rope(B, Hq, Hkv, N, d, rot, interleaved, weights, far):
    g = gen(1)
    q, k = rand(g, B, Hq, N, d, std=3.0), rand(g, B, Hkv, N, d)
    freq = fbs.rope_freqs(rot, 500000.0) if rot else None
    pos = (far + torch.arange(N, device="cuda")[None] + 3 * torch.arange(B, device="cuda")[:, None]).to(torch.int32)
    wq, wk = ((1 + 0.5 * torch.randn(d, generator=g, device="cuda")) if weights else None for _ in range(2))
    a, b = fbs.qk_norm_rope(q, k, freq, positions=pos, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved)
    for x, w, y in ((q, wq, a), (k, wk, b)):
        ref, mag = R.norm_rope(x.double(), w, freq, pos, 1e-5, interleaved)
        # fp64 angles of far positions are themselves off: position * frequency * 2^-52 of a radian
        within(y, ref, 2.0 ** -8 * ref.abs() + (2.0 ** -19 + 2.0 ** -50 * abs(far)) * mag)


def test_norm_rope_outputs_stand_apart():
    """The outputs that a small call makes are tensors of their own: writing one leaves the other, one given output is
    filled and returned, and the empty call gives empty tensors."""
    g = gen(26)
    q, k = rand(g, 2, 3, 5, 64), rand(g, 2, 1, 5, 64)
    freq = fbs.rope_freqs(64)
    a, b = fbs.qk_norm_rope(q, k, freq)
    keep = b.clone()
    a.fill_(7.0)
    assert torch.equal(b, keep) and a.is_contiguous() and b.is_contiguous()
    mine = torch.empty_like(q)
    c, d = fbs.qk_norm_rope(q, k, freq, q_out=mine)
    assert c is mine and torch.equal(d, keep)
    big = rand(g, 1, 8, 2000, 64)
    x, y = fbs.qk_norm_rope(big, big, freq)
    assert torch.equal(x, y) and x.untyped_storage().data_ptr() != y.untyped_storage().data_ptr()


def test_norm_rope_strides_start_and_in_place():
    g = gen(2)
    B, Hq, Hkv, N, d = 2, 6, 2, 50, 128
    q = rand(g, B, N, Hq + 1, d)[:, :, :Hq].transpose(1, 2)      # (B, N, H, d) in memory, padded
    k = rand(g, B, N, Hkv, d).transpose(1, 2)
    freq = fbs.rope_freqs(d)
    pos = (1234 + torch.arange(N, device="cuda"))[None].expand(B, N).to(torch.int32).contiguous()
    a, b = fbs.qk_norm_rope(q, k, freq, positions=pos)
    c, e = fbs.qk_norm_rope(q, k, freq, start=1234)
    assert torch.equal(a, c) and torch.equal(b, e)
    ref, mag = R.norm_rope(q.double(), None, freq, pos, 1e-6, False)
    within(a, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -19 * mag)
    q2, k2 = q.clone(memory_format=torch.preserve_format), k.clone()
    fbs.qk_norm_rope(q2, k2, freq, positions=pos, q_out=q2, k_out=k2)
    assert torch.equal(q2, a) and torch.equal(k2, b)


# ------------------------------------------------------------------------------------------------ tables
def tables_ref(lens, new, free, table, P, N):
    R_, W = table.shape
    table, slots, pos, used = table.clone(), torch.full((R_, N), -1, dtype=torch.int64), torch.full((R_, N), -1, dtype=torch.int32), 0
    for r in range(R_):
        n0, n1 = int(lens[r]), int(lens[r]) + int(new[r])
        for j in range(-(-n0 // P), -(-n1 // P)):
            if j < W:
                table[r, j] = free[used] if used < len(free) else -1
            used += 1
        for i, p in enumerate(range(n0, n1)):
            pos[r, N - int(new[r]) + i] = p
            page = int(table[r, p // P]) if p // P < W else -1
            slots[r, N - int(new[r]) + i] = page * P + p % P if page >= 0 else -1
    return table, slots, pos, lens + new, used


@pytest.mark.parametrize("R_,N,P,top,F,W", [
    (1, 1, 64, 0, 4, 3), (1, 4100, 16, 77, 400, 300), (7, 5, 16, 40, 64, 8), (33, 130, 32, 500, 400, 24),
    (700, 3, 64, 300, 900, 8),        # several requests per CTA
    (9, 40, 16, 100, 11, 12),         # too few free pages
    (5, 1, 256, 1000, 9, 5), (3, 0, 16, 20, 2, 4),
])
def test_cache_tables(R_, N, P, top, F, W):
    g = torch.Generator().manual_seed(R_ * 1000 + N)
    lens = torch.randint(0, top + 1, (R_,), generator=g, dtype=torch.int32)
    new = torch.randint(0, N + 1, (R_,), generator=g, dtype=torch.int32)
    new[0] = N
    free = torch.randperm(5000, generator=g)[:F].to(torch.int32)
    big = torch.randint(0, 5000, (R_, W + 3), generator=g).to(torch.int32)
    want = tables_ref(lens, new, free, big[:, :W], P, N)
    dev = big.cuda()
    slots, pos, kv, used = fbs.cache_tables(lens.cuda(), new.cuda(), free.cuda(), dev[:, :W], P, N)
    assert torch.equal(dev[:, :W].cpu(), want[0]) and torch.equal(dev[:, W:].cpu(), big[:, W:])
    assert torch.equal(slots.cpu(), want[1]) and torch.equal(pos.cpu(), want[2])
    assert torch.equal(kv.cpu(), want[3]) and int(used) == want[4]
    assert fbs.device_status() == 0


def test_cache_tables_reports_bad_requests():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((5, 2), -7, dtype=torch.int32, device="cuda")
    slots, pos, kv, used = fbs.cache_tables(i32(-1, 0, 2 ** 31 - 1, 3, 30), i32(1, 9, 1, 2, 4), i32(5, 6, 7), table, 16, 4)
    assert kv.tolist() == [0, 0, 0, 5, 34] and int(used) == 1
    assert (slots[:3] == -1).all() and (pos[:3] == -1).all()
    assert table[3].tolist() == [-7, -7] and slots[3].tolist() == [-1] * 4   # its page was -7: no slot
    assert slots[4].tolist() == [-1, -1, -1, -1] and pos[4].tolist() == [30, 31, 32, 33]  # page 2 lies past the width
    with pytest.raises(fbs.SpargeError):
        fbs._check(fbs.device_status())
    assert fbs.device_status() == 0


# ------------------------------------------------------------------------------------------- store and load
def values_of(pool, d, slots):
    """K and V of the slots ((B, N), >= 0) in fp64, read by the documented layout."""
    kn, ks, km, vn, vs, vm = R.read_pool(pool, d)
    page = kn.shape[2]
    pick = lambda x: x[slots // page, :, slots % page].transpose(1, 2)  # noqa: E731   (B, H, N, ...)
    return [pick(x) for x in (kn, ks, km, vn, vs, vm)]


def some_slots(g, B, N, page, n_pages, scatter):
    if scatter:
        return torch.randperm(n_pages * page, generator=g, device="cuda")[: B * N].view(B, N)
    per = n_pages // B
    pages = torch.randperm(n_pages, generator=g, device="cuda")[: B * per].view(B, per)
    first = torch.randint(0, page, (B, 1), generator=g, device="cuda")
    at = first + torch.arange(N, device="cuda")[None]
    return (torch.gather(pages, 1, at // page) * page + at % page).contiguous()


@pytest.mark.parametrize("B,H,N,d,page,scatter", [
    (1, 1, 1, 64, 16, False), (5, 8, 1, 128, 64, False), (2, 2, 100, 128, 64, False), (3, 1, 77, 64, 16, False),
    (2, 3, 50, 128, 32, True), (1, 2, 16, 128, 128, False), (1, 1, 700, 64, 256, False), (4, 2, 15, 64, 64, True),
    (2, 2, 4096, 128, 64, False),
])
def test_store_and_load(B, H, N, d, page, scatter):
    g = gen(3)
    n_pages = B * (-(-N // page) + 1) + 2
    k, v = rand(g, B, H, N, d, std=2.0), rand(g, B, N, H, d).transpose(1, 2)
    pool = fbs.cache4_pool(n_pages, page, H, d)
    pool.random_(0, 256, generator=g)
    before = pool.clone()
    slots = some_slots(g, B, N, page, n_pages, scatter)
    fbs.cache4_store(k, v, slots, pool)
    got = values_of(pool, d, slots)
    want = [*R.quantise(k.double()), *R.quantise(v.double())]
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    a, b = fbs.cache4_load(pool, slots)
    assert torch.equal(a, R.dequantise(*want[:3]).float().bfloat16())
    assert torch.equal(b, R.dequantise(*want[3:]).float().bfloat16())
    # every other token is as it was
    other = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    other[slots.flatten()] = False
    rest = other.nonzero().view(1, -1)
    for x, y in zip(values_of(pool, d, rest), values_of(before, d, rest)):
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))


def test_store_edge_values():
    d, page = 128, 64
    k = torch.zeros(1, 1, 8, d, device="cuda")
    k[0, 0, 1] = 3.0                                   # equal values: scale 0
    k[0, 0, 2, :64] = torch.linspace(-1, 1, 64)
    k[0, 0, 2, 64:] = 1e-38 * torch.arange(64)         # scales near the smallest normal
    k[0, 0, 3, 5] = math.inf
    k[0, 0, 4, 70] = math.nan
    k[0, 0, 5, 0], k[0, 0, 5, 1] = 3.3e38, -3.3e38     # a range past fp32
    k[0, 0, 6] = 1e-40                                 # subnormal
    k[0, 0, 7] = torch.arange(d) * -1.5
    k = k.bfloat16()
    pool = fbs.cache4_pool(1, page, 1, d)
    slots = torch.arange(8, device="cuda")[None] * 3
    fbs.cache4_store(k, k, slots, pool)
    a, b = fbs.cache4_load(pool, slots)
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    assert torch.isnan(a[0, 0, 3, :64]).all() and torch.isnan(a[0, 0, 4, 64:]).all()
    assert torch.isfinite(a[0, 0, 3, 64:]).all() and torch.isfinite(a[0, 0, 4, :64]).all()
    assert (a[0, 0, 1] == 3.0).all() and (a[0, 0, 0] == 0).all()
    for t in (2, 7):
        n, s, m = R.quantise(k[0, 0, t].double())
        assert torch.equal(a[0, 0, t], R.dequantise(n, s, m).float().bfloat16())
    assert torch.isfinite(a[0, 0, 5]).all() and torch.isfinite(a[0, 0, 6]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_store_edge_values_in_long_rows(d):
    """Groups without a range, past fp32's range, with infinities and NaN between ordinary ones, in whole records and at
    the ends of rows: codes, scales and minima as defined, NaN only where a group holds one."""
    g = gen(23)
    k, v = rand(g, 1, 3, 70, d), rand(g, 1, 3, 70, d)
    for x in (k, v):
        x[0, 0, ::7] = 3.0
        x[0, 1, 3::9, :64] = 0.0
        x[0, 2, 5::8] *= 1e-36
        x[0, 1, 6, 0], x[0, 1, 6, 1] = 3.3e38, -3.3e38
        x[0, 0, 20, 5], x[0, 2, 69, d - 1], x[0, 1, 40, 33] = math.inf, math.nan, -math.inf
    pool = fbs.cache4_pool(2, 64, 3, d)
    slots = (torch.arange(70, device="cuda")[None] + 25).contiguous()
    fbs.cache4_store(k, v, slots, pool)
    a, b = fbs.cache4_load(pool, slots)
    for x, y in ((k, a), (v, b)):
        groups, back = x.view(1, 3, 70, d // 64, 64), y.reshape(1, 3, 70, d // 64, 64)
        bad = ~torch.isfinite(groups.float()).all(-1)
        assert torch.isnan(back[bad]).all() and torch.isfinite(back[~bad]).all()
        plain = ~bad
        plain[0, 1, 6, 0] = False  # its scale is the one that fp32 can hold
        want = R.dequantise(*R.quantise(torch.where(bad[..., None], torch.zeros_like(groups), groups).reshape(k.shape).double()))
        assert torch.equal(back[plain], want.float().bfloat16().view_as(back)[plain])


def test_loaded_outputs_stand_apart():
    """K and V that a small load makes are tensors of their own; a load of nothing gives empty ones."""
    g = gen(27)
    k, v = rand(g, 2, 1, 3, 64), rand(g, 2, 1, 3, 64)
    pool = fbs.cache4_pool(1, 16, 1, 64)
    slots = torch.arange(6, device="cuda").view(2, 3)
    fbs.cache4_store(k, v, slots, pool)
    a, b = fbs.cache4_load(pool, slots)
    keep = b.clone()
    a.fill_(7.0)
    assert torch.equal(b, keep) and torch.equal(b, R.dequantise(*R.quantise(v.double())).float().bfloat16())
    assert fbs.cache4_load(pool, slots[:0])[1].shape == (0, 1, 3, 64)


@pytest.mark.parametrize("H,d,shift", [(3, 64, 8), (1, 64, 8), (5, 128, 8), (2, 128, 16)])
def test_store_and_load_strided_rows_with_gaps(H, d, shift):
    """Rows that start on 16 but not on 32 bytes (or on 32, with gaps), long rows with padding in front and slots left out in
    the middle; padding rows hold NaN, left-out rows of given outputs keep what they held."""
    g = gen(24)
    B, N, page = 2, 61, 32
    wide = lambda: rand(g, B, N, H, d + shift)[..., shift:].transpose(1, 2)  # noqa: E731
    k, v = wide(), wide()
    slots = torch.stack([torch.arange(N, device="cuda") + 7, torch.arange(N, device="cuda") + 100])
    slots[0, :20] = -1
    slots[1, 30:33] = -4
    k.transpose(1, 2)[slots < 0] = math.nan
    v.transpose(1, 2)[slots < 0] = math.inf
    pool = fbs.cache4_pool(6, page, H, d)
    pool.random_(0, 256, generator=g)
    before = pool.clone()
    fbs.cache4_store(k, v, slots, pool)
    a, b = wide().fill_(9.0), wide().fill_(9.0)
    fbs.cache4_load(pool, slots, a, b)
    a2, b2 = fbs.cache4_load(pool, slots)
    live = slots >= 0
    for x, got, made in ((k, a, a2), (v, b, b2)):
        want = R.dequantise(*R.quantise(x.transpose(1, 2)[live].double())).float().bfloat16()
        assert torch.equal(got.transpose(1, 2)[live], want) and torch.equal(made.transpose(1, 2)[live], want)
        assert (got.transpose(1, 2)[~live] == 9).all() and (made.transpose(1, 2)[~live] == 0).all()
    other = torch.ones(6 * page, dtype=torch.bool, device="cuda")
    other[slots[live]] = False
    rest = other.nonzero().view(1, -1)
    for x, y in zip(values_of(pool, d, rest), values_of(before, d, rest)):
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))


def test_slots_left_out():
    d, page, H = 64, 16, 2
    g = gen(4)
    k, v = rand(g, 2, H, 5, d), rand(g, 2, H, 5, d)
    pool = fbs.cache4_pool(2, page, H, d)
    pool.random_(0, 256, generator=g)
    before = pool.clone()
    slots = torch.tensor([[-1, -1, 0, 1, 2], [-5, 31, 30, -1, 20]], device="cuda")
    fbs.cache4_store(k, v, slots, pool)
    a, b = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    fbs.cache4_load(pool, slots, a, b)
    out = slots < 0
    assert (a.transpose(1, 2)[out] == 9).all() and (b.transpose(1, 2)[out] == 9).all()
    assert not (a.transpose(1, 2)[~out] == 9).all()
    assert fbs.device_status() == 0
    pool.copy_(before)
    past = torch.full_like(slots, 32)
    past[0, 0] = 2 ** 62
    fbs.cache4_store(k, v, past, pool)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    assert torch.equal(pool, before)
    a.fill_(9.0)
    fbs.cache4_load(pool, past, a, b)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG and (a == 9).all()


# -------------------------------------------------------------------------------------- attention over the cache
def filled(g, lens, H, d, page, std=1.0):
    """A pool with the sequences' tokens on shuffled pages and rubbish (NaN scales) everywhere else; its tables."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
    pool = fbs.cache4_pool(sum(need) + 3, page, H, d)
    pool.fill_(255)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
        if n:
            k, v = rand(g, 1, H, n, d, std=std), rand(g, 1, H, n, d)
            k[..., 3] += 4.0
            v[:, :, n // 2:] *= 30.0                    # scales that grow along the sequence
            t = torch.arange(n, device="cuda")
            fbs.cache4_store(k, v, (table[b].long()[t // page] * page + t % page)[None].contiguous(), pool)
    return pool, table


def check_cache_attn(q, pool, table, lens, out, d, window=0, sinks=0, scale=0.0, rows=None):
    page = 16 * pool.shape[2]
    kn, ks, km, vn, vs, vm = R.read_pool(pool, d)
    K, V, E = R.dequantise(kn, ks, km), R.dequantise(vn, vs, vm), R.dequantise(vn, vs, torch.zeros_like(vm))
    for b, n in enumerate(lens):
        if rows is not None and b not in rows:
            continue
        Nq = q.shape[2]
        if n == 0:
            assert (out[b] == 0).all()
            continue
        t = torch.arange(n, device="cuda")
        seq = lambda x: x[table[b].long()[t // page], :, t % page].transpose(0, 1)  # noqa: E731
        k, v, e = seq(K), seq(V), seq(E)
        pos = n - Nq + torch.arange(Nq, device="cuda")
        o, a, x = R.attention(q[b].double(), k, v, pos, window, sinks, scale or d ** -0.5, e)
        vmax = torch.nan_to_num(v).abs().amax() + torch.nan_to_num(e).abs().amax()
        within(out[b], o, 2.0 ** -8 * o.abs() + 2.0 ** -11 * a + 2 * (2.0 ** -16 * x + 2.0 ** -20) * vmax)


@pytest.mark.parametrize("Hq,Hkv,Nq,d,page,lens,window,sinks", [
    (1, 1, 1, 64, 16, [1], 0, 0),
    (4, 1, 1, 128, 64, [1, 0, 64, 65, 15, 16, 17], 0, 0),
    (32, 8, 1, 128, 64, [4096 + 7], 0, 0),
    (8, 8, 1, 64, 32, [300, 5, 1000], 0, 0),
    (8, 1, 1, 128, 16, [777], 0, 0),                 # 8 rows
    (16, 1, 1, 128, 128, [500, 33], 0, 0),           # 16 rows
    (6, 2, 5, 64, 64, [2, 5, 700], 0, 0),            # 15 rows; a sequence shorter than its queries
    (10, 2, 7, 128, 256, [900, 6], 0, 0),            # 35 rows: three row tiles
    (32, 8, 1, 128, 64, [4096 + 7, 10], 100, 4),
    (8, 2, 4, 64, 16, [2000, 50, 51, 3], 48, 37),
    (4, 2, 3, 128, 32, [1500, 129], 1, 0),           # a window of the query alone
    (4, 4, 1, 128, 64, [700], 10000, 3),             # a window longer than the sequence
    (2, 1, 2, 64, 64, [5000], 64, 64),
])
def test_cache_attn(Hq, Hkv, Nq, d, page, lens, window, sinks):
    g = gen(5)
    pool, table = filled(g, lens, Hkv, d, page)
    q = rand(g, len(lens), Hq, Nq, d)
    q[0, 0, 0] = 0.0
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = fbs.cache4_attn(q, pool, table, kv, window=window, sinks=sinks)
    check_cache_attn(q, pool, table, lens, out, d, window, sinks)


def test_cache_attn_many_ragged_sequences():
    """More sequences than threads that sum their lengths, many of them empty or one token long."""
    g = gen(6)
    lens = [(7 * i * i) % 211 if i % 3 else 0 for i in range(300)]
    pool, table = filled(g, lens, 2, 64, 16)
    q = rand(g, len(lens), 4, 1, 64)
    out = fbs.cache4_attn(q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check_cache_attn(q, pool, table, lens, out, 64)


def test_cache_attn_strides_scale_and_peaked_scores():
    g = gen(7)
    lens, d = [1000, 333], 128
    pool, table = filled(g, lens, 2, d, 64, std=4.0)
    wide = torch.full((2, table.shape[1] + 5), 77777, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = rand(g, 2, 1, 9, d, std=8.0).transpose(1, 2)[:, :8]      # strides of (B, N, H, d)
    out = torch.empty(2, 1, 8, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = fbs.cache4_attn(q, pool, wide[:, :table.shape[1]], kv, scale=0.3, out=out)
    assert got is out
    check_cache_attn(q, pool, table, lens, out, d, scale=0.3)


def test_cache_attn_bad_pages_and_lengths():
    """A page outside the pool is left out (as if its tokens were not there) and reported; lengths are held within
    the table."""
    g = gen(8)
    d, page = 64, 16
    pool, table = filled(g, [64, 64], 1, d, page)
    q = rand(g, 2, 2, 1, d)
    kv = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
    good = fbs.cache4_attn(q, pool, table, kv)
    bad = table.clone()
    bad[0, 1], bad[0, 2] = -1, pool.shape[0]
    got = fbs.cache4_attn(q, pool, bad, kv)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    assert torch.equal(got[1], good[1])
    short = table.clone()
    short[0, 1] = table[0, 3]
    check = fbs.cache4_attn(q, pool, short, torch.tensor([32, 64], dtype=torch.int32, device="cuda"))
    assert (got[0].float() - check[0].float()).abs().max() <= 2.0 ** -6 * check[0].float().abs().max()
    long = fbs.cache4_attn(q, pool, table, torch.tensor([2 ** 31 - 1, -3], dtype=torch.int32, device="cuda"))
    assert torch.equal(long[0], good[0]) and (long[1] == 0).all()
    assert fbs.device_status() == 0


def test_cache_attn_poison_outside_the_window():
    """NaN keys and values (a group that held an infinity) that no query sees change nothing; seen, they show."""
    g = gen(9)
    d, n = 128, 400
    pool, table = filled(g, [n], 1, d, 64)
    q = rand(g, 1, 4, 1, d)
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    good = fbs.cache4_attn(q, pool, table, kv, window=50, sinks=2)
    inf = torch.full((1, 1, 3, d), math.inf, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([2, 349, 200], device="cuda")
    fbs.cache4_store(inf, inf, (table[0].long()[at // 64] * 64 + at % 64)[None].contiguous(), pool)
    assert torch.equal(fbs.cache4_attn(q, pool, table, kv, window=50, sinks=2), good)
    assert torch.isnan(fbs.cache4_attn(q, pool, table, kv, window=51, sinks=2)).all()


# -------------------------------------------------------------------------------------------- window attention
def check_window(q, k, v, out, window, sinks, scale=0.0, decode=False):
    B, Hq, Nq, d = q.shape
    Nk = k.shape[2]
    for b in range(B):
        pos = Nk - Nq + torch.arange(Nq, device="cuda")
        o, a, x = R.attention(q[b].double(), k[b].double(), v[b].double(), pos, window, sinks, scale or d ** -0.5)
        p = 2.0 ** -16 if decode else 2.0 ** -11
        within(out[b], o, 2.0 ** -8 * o.abs() + p * a + 2 * (2.0 ** -16 * x + 2.0 ** -20) * v[b].double().abs().amax())


@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nk,d,window,sinks,decode", [
    (1, 1, 1, 1, 1, 64, 1, 0, False),
    (1, 2, 1, 128, 128, 128, 128, 0, False),
    (1, 4, 2, 300, 300, 64, 70, 5, False),
    (2, 3, 1, 257, 1000, 128, 64, 1, False),
    (1, 2, 2, 1000, 1000, 64, 1, 0, False),        # each query sees itself
    (1, 2, 2, 700, 700, 128, 129, 64, False),
    (1, 2, 1, 500, 900, 64, 333, 100, False),
    (1, 2, 2, 640, 640, 128, 5000, 3, False),      # a window longer than the keys: causal
    (1, 2, 1, 2049, 2049, 128, 511, 4, False),
    (1, 4, 1, 1, 500, 128, 64, 4, False),          # few queries, few blocks
    (1, 2, 1, 700, 4000, 128, 2000, 100, False),   # long windows
    (2, 4, 2, 1500, 2500, 128, 1700, 4, False),
    (1, 2, 2, 2000, 2000, 64, 1900, 70, False),
    (1, 16, 1, 333, 700, 64, 200, 5, False),       # tiles of 8 queries of 16 heads
    (2, 12, 1, 77, 1000, 128, 100, 0, False),      # of 32 queries of 4
    (1, 20, 10, 300, 300, 64, 47, 1, False),       # of 64 queries of 2
    (1, 32, 1, 9, 200, 64, 30, 0, False),          # two groups of 16 heads
    (1, 6, 1, 130, 1400, 128, 1270, 3, False),     # 23 and 24 blocks a query block
    (1, 6, 1, 130, 1500, 128, 1330, 3, False),
    (2, 8, 2, 1, 5000, 128, 2100, 4, True),        # few rows: tiles of 8 or 16
    (1, 8, 1, 7, 4001, 64, 2500, 0, True),
    (3, 4, 4, 1, 2300, 64, 10000, 0, True),
    (1, 16, 2, 16, 9000, 128, 3000, 130, True),
])
def test_window_attn(B, Hq, Hkv, Nq, Nk, d, window, sinks, decode):
    g = gen(10)
    q, k, v = rand(g, B, Hq, Nq, d), rand(g, B, Hkv, Nk, d), rand(g, B, Hkv, Nk, d)
    k[:, :, :sinks] *= 2.0
    out = fbs.window_attn(q, k, v, window, sinks)
    check_window(q, k, v, out, window, sinks, decode=decode)


def test_window_attn_strides_scale_and_workspace():
    g = gen(11)
    q, k, v = (rand(g, 1, 400, h, 64).transpose(1, 2) for h in (4, 2, 2))
    out = torch.full((1, 400, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    ws = torch.empty(fbs.workspace_bytes(fbs.SPARGE_OP_WINDOW_ATTN, 1, 4, 2, 400, 64), dtype=torch.uint8, device="cuda")
    fbs.window_attn(q, k, v, 90, 3, scale=0.5, out=out, ws=ws)
    check_window(q, k, v, out, 90, 3, scale=0.5)


def test_window_attn_is_causal_attention_under_a_long_window():
    """Against the block-sparse attention without a mask; both are within their tolerance of the definition."""
    g = gen(12)
    q, k, v = rand(g, 1, 4, 900, 128), rand(g, 1, 2, 900, 128), rand(g, 1, 2, 900, 128)
    check_window(q, k, v, fbs.window_attn(q, k, v, 900), 900, 0)
    check_window(q, k, v, fbs.block_sparse_attn(q, k, v, None, -math.inf, True), 900, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_window_attn_climbing_scores(d):
    """Scores that climb by more than the rescaling threshold from block to block and within a step, so O, the row sum
    and the P of a step's first columns are scaled down again and again; and a peak at the window's end."""
    g = gen(15)
    N = 700
    u = torch.randn(d, generator=g, device="cuda")
    u = u / u.norm()
    ramp = torch.arange(N, device="cuda") // 32 * 0.6
    q = (8.0 * u + 0.1 * torch.randn(1, 2, N, d, generator=g, device="cuda")).bfloat16()
    k = (ramp[:, None] * u * math.sqrt(d) + 0.1 * torch.randn(1, 1, N, d, generator=g, device="cuda")).bfloat16()
    v = rand(g, 1, 1, N, d)
    check_window(q, k, v, fbs.window_attn(q, k, v, 300, 5), 300, 5)
    k2 = k.flip(2).contiguous()
    check_window(q, k2, v, fbs.window_attn(q, k2, v, 300, 5), 300, 5)


def test_window_attn_beside_other_attention():
    """Window attention at both head dims and the block-sparse attention on three streams at once, all of them with
    accumulators in tensor memory: the same bits as one after another."""
    g = gen(25)
    a = [rand(g, 1, h, 2500, 64) for h in (16, 4, 4)]
    b = [rand(g, 1, h, 2500, 128) for h in (8, 2, 2)]
    calls = [lambda: fbs.window_attn(*a, 500, 4), lambda: fbs.window_attn(*b, 300, 4), lambda: fbs.block_sparse_attn(*b, None, -math.inf, True)]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], [], []]
    for _ in range(10):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    for i in range(3):
        assert all(torch.equal(x, want[i]) for x in got[i])


# ------------------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_serving_steps_together(window, sinks):
    """A prefill chunk and decoding steps of a ragged batch: tables, norm and rotation, store, attention, each
    step's output against attention over everything stored so far; padding places change nothing."""
    g = gen(13)
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    freq = fbs.rope_freqs(d)
    pool = fbs.cache4_pool(64, page, Hkv, d)
    pool.fill_(255)
    table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(64, generator=g, device="cuda").to(torch.int32)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = [torch.empty(Hkv, 0, d, dtype=torch.float64, device="cuda") for _ in range(2 * B)]
    for step, new in enumerate([[20, 1, 7], [1, 1, 1], [0, 1, 1], [3, 2, 3], [1, 1, 1]]):
        N = max(new)
        add = torch.tensor(new, dtype=torch.int32, device="cuda")
        slots, pos, kv, used = fbs.cache_tables(lens, add, free, table, page, N)
        free = free[int(used):].contiguous()
        x = [rand(g, B, h, N, d) for h in (Hq, Hkv, Hkv)]
        q, k = fbs.qk_norm_rope(x[0], x[1], freq, positions=pos)
        fbs.cache4_store(k, x[2], slots, pool)
        out = fbs.cache4_attn(q, pool, table, kv, window=window, sinks=sinks)
        for b, n in enumerate(new):
            if n == 0:
                continue
            kept[2 * b] = torch.cat([kept[2 * b], R.dequantise(*R.quantise(k[b, :, N - n:].double()))], 1)
            kept[2 * b + 1] = torch.cat([kept[2 * b + 1], R.dequantise(*R.quantise(x[2][b, :, N - n:].double()))], 1)
            total = kept[2 * b].shape[1]
            p = total - n + torch.arange(n, device="cuda")
            o, a, s = R.attention(q[b, :, N - n:].double(), kept[2 * b], kept[2 * b + 1], p, window, sinks, d ** -0.5)
            vmax = kept[2 * b + 1].abs().amax()
            # |scale code| = |v - minimum| is at most twice the largest |v|
            within(out[b, :, N - n:], o, 2.0 ** -8 * o.abs() + 2 * (2.0 ** -11 + 2.0 ** -16 * s + 2.0 ** -20) * 2 * vmax)
        lens = kv
    assert lens.tolist() == [25, 6, 13] and fbs.device_status() == 0


def test_cache_attn_long_chunk_of_queries():
    """Many row tiles: 1200 query rows per KV head, in tiles of 16."""
    g = gen(16)
    lens, d = [777, 300], 128
    pool, table = filled(g, lens, 2, d, 32)
    q = rand(g, 2, 8, 300, d)
    out = fbs.cache4_attn(q, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), window=200, sinks=3)
    check_cache_attn(q, pool, table, lens, out, d, 200, 3)


def test_cache_attn_shared_pages_and_repeated_calls():
    """Two sequences on the same pages (a shared prefix) and the same sequence twice; calls give the same bits each time."""
    g = gen(17)
    d = 64
    pool, table = filled(g, [600], 2, d, 16)
    table = table.expand(3, -1)
    lens = [600, 333, 600]
    q = rand(g, 1, 4, 1, d).expand(3, -1, -1, -1).contiguous()
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = fbs.cache4_attn(q, pool, table.contiguous(), kv)
    check_cache_attn(q, pool, table, lens, out, d)
    # the cut into shares differs between the two, so their sums may round differently
    assert (out[0].float() - out[2].float()).abs().max() <= 2.0 ** -7 * out[0].float().abs().max()
    for _ in range(3):
        assert torch.equal(fbs.cache4_attn(q, pool, table.contiguous(), kv), out)


def test_pool_past_32_bits():
    """Pages past 4 GiB of pool: stored, read back and attended to."""
    g = gen(18)
    d, page, H = 128, 256, 8
    per = page * H * (d + d // 8)
    pool = torch.empty((5 << 30) // per, H, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
    n = pool.shape[0]
    assert n * per > 1 << 32
    table = torch.tensor([[n - 1, 3, n - 2]], dtype=torch.int32, device="cuda")
    k, v = rand(g, 1, H, 600, d), rand(g, 1, H, 600, d)
    t = torch.arange(600, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page)[None].contiguous()
    fbs.cache4_store(k, v, slots, pool)
    a, b = fbs.cache4_load(pool, slots)
    assert torch.equal(a, R.dequantise(*R.quantise(k.double())).float().bfloat16())
    q = rand(g, 1, 16, 1, d)
    out = fbs.cache4_attn(q, pool, table, torch.tensor([600], dtype=torch.int32, device="cuda"))
    kk, vv = (R.dequantise(*R.quantise(x.double()))[0] for x in (k, v))
    o, _, x = R.attention(q[0].double(), kk, vv, torch.tensor([599], device="cuda"), 0, 0, d ** -0.5)
    within(out[0], o, 2.0 ** -8 * o.abs() + 2 * (2.0 ** -11 + 2.0 ** -16 * x + 2.0 ** -20) * 2 * vv.abs().amax())
    assert fbs.device_status() == 0


def test_calls_on_two_streams_at_once():
    g = gen(19)
    d = 128
    pools = [filled(g, [3000 + 100 * i, 70], 2, d, 64) for i in range(2)]
    qs = [rand(g, 2, 8, 1, d) for _ in range(2)]
    kv = [torch.tensor([3000 + 100 * i, 70], dtype=torch.int32, device="cuda") for i in range(2)]
    kw, qw = rand(g, 1, 2, 5000, d), rand(g, 1, 8, 1, d)
    want = [fbs.cache4_attn(q, p, t, n) for q, (p, t), n in zip(qs, pools, kv)]
    want_w = fbs.window_attn(qw, kw, kw, 3000, 4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((fbs.cache4_attn(qs[i], *pools[i], kv[i]), fbs.window_attn(qw, kw, kw, 3000, 4)))
    torch.cuda.synchronize()
    for i in range(2):
        for a, w in got[i]:
            assert torch.equal(a, want[i]) and torch.equal(w, want_w)


@pytest.mark.parametrize("Nq", [1, 3, 200])
def test_window_attn_ignores_keys_that_no_query_sees(Nq):
    """NaN and infinities in keys and values in front of the window (a ring buffer's leftovers) change nothing."""
    g = gen(20)
    q, k, v = rand(g, 1, 4, Nq, 64), rand(g, 1, 2, 1000, 64), rand(g, 1, 2, 1000, 64)
    good = fbs.window_attn(q, k, v, 333, 5)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, 5:1000 - Nq - 333 + 1] = math.nan
    v2[:, :, 5:1000 - Nq - 333 + 1] = math.inf
    v2[:, :, 7] = v2[:, :, 1000 - Nq - 333] = math.nan
    assert torch.equal(fbs.window_attn(q, k2, v2, 333, 5), good)


def test_empty_calls():
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = fbs.cache4_pool(2, 16, 2, 64)
    assert fbs.cache4_attn(e(0, 4, 1, 64), pool, i32(0, 3), i32(0)).shape == (0, 4, 1, 64)
    assert fbs.cache4_attn(e(2, 4, 0, 64), pool, i32(2, 3), i32(2)).shape == (2, 4, 0, 64)
    assert (fbs.cache4_attn(torch.ones_like(e(2, 4, 1, 64)), pool, i32(2, 0), torch.full((2,), 9, dtype=torch.int32, device="cuda")) == 0).all()
    assert fbs.window_attn(e(1, 4, 0, 64), e(1, 2, 5, 64), e(1, 2, 5, 64), 3).shape == (1, 4, 0, 64)
    a, b = fbs.qk_norm_rope(e(2, 4, 0, 64), e(2, 2, 0, 64), fbs.rope_freqs(64))
    assert a.shape == (2, 4, 0, 64) and b.shape == (2, 2, 0, 64)
    fbs.cache4_store(e(2, 2, 0, 64), e(2, 2, 0, 64), torch.empty(2, 0, dtype=torch.int64, device="cuda"), pool)
    assert fbs.cache4_load(pool, torch.empty(2, 0, dtype=torch.int64, device="cuda"))[0].shape == (2, 2, 0, 64)
    slots, pos, kv, used = fbs.cache_tables(i32(0), i32(0), i32(0), i32(0, 3), 16, 4)
    assert slots.shape == (0, 4) and int(used) == 0
    torch.cuda.synchronize()
    assert fbs.device_status() == 0


def test_calls_refuse_what_they_cannot_take():
    g = gen(21)
    q, k = rand(g, 1, 4, 8, 64), rand(g, 1, 2, 8, 64)
    pool = fbs.cache4_pool(4, 16, 2, 64)
    slots = torch.zeros(1, 8, dtype=torch.int64, device="cuda")
    table, kv = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for call, err in ((lambda: fbs.window_attn(q.float(), k, k, 4), TypeError), (lambda: fbs.window_attn(q, k.cpu(), k, 4), ValueError),
                      (lambda: fbs.window_attn(q, k, k, 0), fbs.SpargeError), (lambda: fbs.window_attn(q.transpose(2, 3), k, k, 4), TypeError),
                      (lambda: fbs.window_attn(q, k, k, 4, ws=torch.empty(16, dtype=torch.uint8, device="cuda")), fbs.SpargeError),
                      (lambda: fbs.qk_norm_rope(q, k, fbs.rope_freqs(64).float()), TypeError),
                      (lambda: fbs.qk_norm_rope(q, k, fbs.rope_freqs(64), positions=torch.zeros(8, dtype=torch.int32, device="cuda")), TypeError),
                      (lambda: fbs.qk_norm_rope(q, k, fbs.rope_freqs(64), q_weight=torch.ones(32, device="cuda")), TypeError),
                      (lambda: fbs.qk_norm_rope(q, k, fbs.rope_freqs(24)), fbs.SpargeError),
                      (lambda: fbs.cache4_store(k, k, slots.int(), pool), TypeError), (lambda: fbs.cache4_store(k, k, slots[:, :7], pool), TypeError),
                      (lambda: fbs.cache4_store(q, q, slots, pool), fbs.SpargeError), (lambda: fbs.cache4_store(k, k, slots, pool[..., :100]), TypeError),
                      (lambda: fbs.cache4_load(pool, slots, k_out=k), ValueError),
                      (lambda: fbs.cache4_attn(q, pool, table.long(), kv), TypeError), (lambda: fbs.cache4_attn(q, pool, table, kv.long()), TypeError),
                      (lambda: fbs.cache4_attn(q, pool, table.expand(2, -1), kv), TypeError),
                      (lambda: fbs.cache4_attn(q, pool, table, kv, sinks=3), fbs.SpargeError),
                      (lambda: fbs.cache_tables(kv, kv, kv, table, 16, -1), ValueError), (lambda: fbs.cache_tables(kv, kv.cpu(), kv, table, 16, 1), ValueError),
                      (lambda: fbs.cache_tables(kv, kv, kv, table, 24, 1), fbs.SpargeError), (lambda: fbs.cache4_pool(4, 20, 2, 64), ValueError)):
        with pytest.raises(err):
            call()
    assert fbs.device_status() == 0


def test_tables_outputs_stand_apart():
    """Outputs that the call makes hold their own values, mixed with given ones too."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want = ([[-1, 5 * 16], [7 * 16, 7 * 16 + 1]], [[-1, 16], [0, 1]], [17, 2], [2])
    for given in ((), (0,), (1, 3), (2,)):
        out = [torch.empty(2, 2, dtype=torch.int64, device="cuda"), i32(0, 0, 0, 0).view(2, 2), i32(0, 0), i32(0)]
        table = i32(3, -9, -9, -9).view(2, 2)
        got = fbs.cache_tables(i32(16, 0), i32(1, 2), i32(5, 7), table, 16, 2, *[o if i in given else None for i, o in enumerate(out)])
        assert tuple(x.tolist() for x in got) == want and table.tolist() == [[3, 5], [7, -9]]
        assert all(got[i] is out[i] for i in given)
        for i, x in enumerate(got):  # writing one changes no other
            x.fill_(-77)
            assert all(y.tolist() == want[j] for j, y in enumerate(got) if j > i)


def test_capture_over_two_streams():
    """Calls on a side stream that forks off the captured one and joins it again, behind kernels, copies and events: the
    graph's replays give what the calls give one after another."""
    g = gen(22)
    d = 64
    pool, table = filled(g, [500, 77], 2, d, 16)
    kv = torch.tensor([500, 77], dtype=torch.int32, device="cuda")
    q, k = rand(g, 2, 4, 1, d), rand(g, 2, 2, 1, d)
    src = rand(g, 2, 4, 1, d)
    freq = fbs.rope_freqs(d)

    def step(s, side):
        q.copy_(src)
        side.wait_stream(s)
        with torch.cuda.stream(side):
            n0, _ = fbs.qk_norm_rope(q, k, freq, start=7)
            o0 = fbs.cache4_attn(n0, pool, table, kv)
        n1, _ = fbs.qk_norm_rope(q, k, freq, start=9)
        o1 = fbs.cache4_attn(n1, pool, table, kv, window=50, sinks=2)
        s.wait_stream(side)
        n2, _ = fbs.qk_norm_rope(o0, k, freq)
        return o0, o1, fbs.cache4_attn(n2 + o1, pool, table, kv)

    s, side = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(s, side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step(s, side)
    torch.cuda.synchronize()
    for _ in range(5):
        src.copy_(rand(g, 2, 4, 1, d))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        a = []
        n0, _ = fbs.qk_norm_rope(src, k, freq, start=7)
        a.append(fbs.cache4_attn(n0, pool, table, kv))
        n1, _ = fbs.qk_norm_rope(src, k, freq, start=9)
        a.append(fbs.cache4_attn(n1, pool, table, kv, window=50, sinks=2))
        n2, _ = fbs.qk_norm_rope(a[0], k, freq)
        a.append(fbs.cache4_attn(n2 + a[1], pool, table, kv))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, out))


def test_a_captured_step_replays():
    """Store and attention of a step captured into a graph, replayed on new inputs in place, on a stream of its own."""
    g = gen(14)
    lens, d, page = [200, 90], 128, 64
    pool, table = filled(g, lens, 2, d, page)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = rand(g, 2, 4, 1, d), rand(g, 2, 2, 1, d), rand(g, 2, 2, 1, d)
    last = kv.long() - 1
    slots = (table.long().gather(1, (last // page)[:, None]) * page + (last % page)[:, None]).contiguous()
    out = torch.empty_like(q)
    kw = torch.randn(2, 1, 300, d, generator=g, device="cuda").bfloat16()
    qw = torch.randn(2, 1, 300, d, generator=g, device="cuda").bfloat16()

    def step():
        fbs.cache4_store(k, v, slots, pool)
        fbs.cache4_attn(q, pool, table, kv, out=out)
        return fbs.window_attn(qw, kw, kw, 60, 2)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            w = step()
    torch.cuda.synchronize()
    for i in range(3):
        q.copy_(rand(g, 2, 4, 1, d))
        k.copy_(rand(g, 2, 2, 1, d))
        kw.copy_(rand(g, 2, 1, 300, d))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        again, w1 = out.clone(), w.clone()
        w2 = step()
        assert torch.equal(again, out) and torch.equal(w1, w2)
        check_cache_attn(q, pool, table, lens, out, d)
