"""The serving operators where values, masks and sizes reach their ends, against fp64 definitions.

Tolerances of the cache attention, per output channel: half a bf16 step of the result (2^-8); P times the scale in f16
(2^-11) and subnormal below 2^-14 while a row's largest stays at 2^3 or above (2^-28 of the largest for each of n
tokens' codes up to 15); scores are fp32 sums of d <= 128 products, off by at most 2^-16 of sum |q||k| scale, and with the
exponent's own error (2^-20) they move each P by that share of itself, before and after the division by the sum."""
import math

import pytest
import torch

import free_block_sparse_gb300 as fbs
import serving_ref as R
from test_gpu_serving import filled, gen, rand, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbs.lib()
    assert torch.cuda.is_available()
    yield
    torch.cuda.synchronize()
    assert fbs.device_status() == 0


# ------------------------------------------------------------------------------ values of uneven size in the cache
def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def store_at(pool, table, t, k, v):
    """Stores k and v (1, H, len(t), d) as tokens t of the sequence on table's first row."""
    page = 16 * pool.shape[2]
    t = torch.as_tensor(t, device="cuda")
    fbs.cache4_store(k, v, (table[0].long()[t // page] * page + t % page)[None].contiguous(), pool)


def check_channels(q, pool, table, n, out, d, window=0, sinks=0):
    """One sequence; the tolerance of every channel from what this row and channel sum up."""
    page = 16 * pool.shape[2]
    t = torch.arange(n, device="cuda")
    kn, ks, km, vn, vs, vm = (x[table[0].long()[t // page], :, t % page].transpose(0, 1) for x in R.read_pool(pool, d))
    k, v, e = R.dequantise(kn, ks, km), R.dequantise(vn, vs, vm), R.dequantise(vn, vs, torch.zeros_like(vm))
    Nq = q.shape[2]
    pos = n - Nq + torch.arange(Nq, device="cuda")
    o, a, x = R.attention(q[0].double(), k, v, pos, window, sinks, d ** -0.5, e)
    _, av, _ = R.attention(q[0].double(), k, v, pos, window, sinks, d ** -0.5, v)
    # P s, summed in place of its maximum, per channel group
    s = vs.repeat_interleave(64, -1)
    _, top, _ = R.attention(q[0].double(), k, v, pos, window, sinks, d ** -0.5, s)
    within(out[0], o, 2.0 ** -8 * o.abs() + 2.0 ** -11 * a + 15 * n * 2.0 ** -28 * top + 2 * (2.0 ** -16 * x + 2.0 ** -20) * (av + a))


SHAPES = [(2, 1, 64), (8, 1, 128), (4, 4, 64), (3, 5, 128)]  # heads of one KV head, queries, d: 8 and 16 rows


@pytest.mark.parametrize("power", [16, 20, 24, 30, 60])
@pytest.mark.parametrize("Hq,Nq,d", SHAPES)
def test_hidden_values_of_any_size_change_nothing(Hq, Nq, d, power):
    """Finite values between the first tokens and the window, in records that hold visible tokens too: the same bits."""
    g = gen(40)
    n = 400
    pool, table = filled(g, [n], 1, d, 64)
    q, kv = rand(g, 1, Hq, Nq, d), i32(n)
    good = fbs.cache4_attn(q, pool, table, kv, window=50, sinks=2)
    k, v = rand(g, 1, 1, 4, d), rand(g, 1, 1, 4, d, std=2.0 ** power)
    store_at(pool, table, [2, 15, 337, 344], k, v)
    assert torch.equal(fbs.cache4_attn(q, pool, table, kv, window=50, sinks=2), good)
    check_channels(q, pool, table, n, good, d, 50, 2)


@pytest.mark.parametrize("power", [0, 16, 24, 30])
@pytest.mark.parametrize("Hq,d", [(2, 64), (5, 128)])
def test_values_that_only_the_last_query_sees(Hq, d, power):
    """The last token is hidden from the other queries of its tile: their rows keep their bits."""
    g = gen(41)
    n, Nq = 300, 3
    pool, table = filled(g, [n], 1, d, 32)
    q, kv = rand(g, 1, Hq, Nq, d), i32(n)
    good = fbs.cache4_attn(q, pool, table, kv)
    store_at(pool, table, [n - 1], rand(g, 1, 1, 1, d), rand(g, 1, 1, 1, d, std=2.0 ** power))
    got = fbs.cache4_attn(q, pool, table, kv)
    assert torch.equal(got[:, :, :-1], good[:, :, :-1])
    check_channels(q, pool, table, n, got, d)


@pytest.mark.parametrize("power", [12, 20, 24, 30, 40])
@pytest.mark.parametrize("at", [0, 3, 200, 298])
@pytest.mark.parametrize("Hq,Nq,d", SHAPES)
def test_large_values_of_improbable_tokens(Hq, Nq, d, at, power):
    """A token that every query sees with a probability of about 2^-30 and values up to 2^40 times the others': the others'
    share of the result stays as exact as without it."""
    g = gen(42)
    n = 300
    pool, table = filled(g, [n], 1, d, 16)
    q = (1 + 0.25 * torch.randn(1, Hq, Nq, d, generator=g, device="cuda")).bfloat16()
    k, v = rand(g, 1, 1, 1, d), rand(g, 1, 1, 1, d, std=2.0 ** power)
    k[:] = -20.0 * d ** -0.5
    store_at(pool, table, [at], k, v)
    check_channels(q, pool, table, n, fbs.cache4_attn(q, pool, table, i32(n)), d)


@pytest.mark.parametrize("power", [16, 24, 30])
@pytest.mark.parametrize("Hq,Nq", [(8, 1), (4, 4)])
def test_large_values_in_one_channel_group(Hq, Nq, power):
    """Channels 64 to 127 of a few tokens 2^16 and more times the rest: channels 0 to 63 stay as exact as without them."""
    g = gen(43)
    n, d = 300, 128
    pool, table = filled(g, [n], 1, d, 64)
    q = rand(g, 1, Hq, Nq, d)
    k, v = rand(g, 1, 1, 3, d), rand(g, 1, 1, 3, d)
    v[..., 64:] *= 2.0 ** power
    store_at(pool, table, [1, 100, 299], k, v)
    check_channels(q, pool, table, n, fbs.cache4_attn(q, pool, table, i32(n)), d)


@pytest.mark.parametrize("std", [2.0 ** -60, 2.0 ** -20, 2.0 ** 40])
@pytest.mark.parametrize("Hq,Nq,d", SHAPES)
def test_scores_that_climb_past_a_large_value(Hq, Nq, d, std):
    """The first token has values 2^30 times the others', and scores climb by 100 behind it, so that its part fades; values
    of any size as a whole."""
    g = gen(44)
    n = 400
    pool, table = filled(g, [n], 1, d, 64)
    q = (1 + 0.1 * torch.randn(1, Hq, Nq, d, generator=g, device="cuda")).bfloat16()
    k, v = rand(g, 1, 1, n, d, std=0.1), rand(g, 1, 1, n, d, std=std)
    k += (torch.arange(n, device="cuda") * (100.0 / n) * d ** -0.5)[:, None].bfloat16()
    v[:, :, 0] *= 2.0 ** 30
    store_at(pool, table, range(n), k, v)
    check_channels(q, pool, table, n, fbs.cache4_attn(q, pool, table, i32(n)), d)


# ----------------------------------------------------------------------------------------- calls one behind another
@pytest.mark.parametrize("d,page,Nq", [(128, 64, 1), (64, 16, 4)])
def test_steps_without_a_pause(d, page, Nq):
    """Tables, norm and rotation, store, attention and window attention enqueued one behind another for many steps, every call
    on what the one in front of it writes into the same buffers: the bits of a run that waits after every call."""
    B, Hq, Hkv, steps, W = 5, 8, 2, 40, 40
    g = gen(45)
    x = [rand(g, steps, B, Hq, Nq, d), rand(g, steps, B, Hkv, Nq, d), rand(g, steps, B, Hkv, Nq, d)]
    new = torch.randint(0, Nq + 1, (steps, B), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.randperm(B * W, generator=g, device="cuda").to(torch.int32)
    freq = fbs.rope_freqs(d)

    def run(wait):
        pause = torch.cuda.synchronize if wait else lambda: None
        pool = fbs.cache4_pool(B * W, page, Hkv, d)
        table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        lens = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2)]
        slots = torch.empty(B, Nq, dtype=torch.int64, device="cuda")
        pos, used = torch.empty(B, Nq, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        q, k, o = (torch.empty(B, h, Nq, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hq))
        free = ids.clone()
        outs = []
        for i in range(steps):
            a, b = lens[i % 2], lens[1 - i % 2]
            fbs.cache_tables(a, new[i], free, table, page, Nq, slots=slots, positions=pos, kv_lens=b, used=used)
            pause()
            fbs.qk_norm_rope(x[0][i], x[1][i], freq, positions=pos, q_out=q, k_out=k)
            pause()
            fbs.cache4_store(k, x[2][i], slots, pool)
            pause()
            fbs.cache4_attn(q, pool, table, b, out=o)
            pause()
            fbs.qk_norm_rope(o, k, freq, start=i, q_out=o, k_out=k)
            pause()
            outs.append(fbs.window_attn(o, k, k, 3, 1))
            pause()
            kk, vv = fbs.cache4_load(pool, slots)
            pause()
            outs += [o.clone(), kk, vv, slots.clone(), b.clone()]
            free = torch.roll(free, -B)        # the next step's pages
            pause()
        torch.cuda.synchronize()
        return outs

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)) for x, y in zip(run(False), want))


# ---------------------------------------------------------------------------------- window attention, values of any size
def check_window_values(q, k, v, out, window, sinks, channels=slice(None)):
    """Tolerance: half a bf16 step; P in f16 (2^-11), with up to 128 rows per KV head in two bf16 (2^-16); above that a copied
    value is off by 2^-19 of the largest of its head; scores as in the cache attention, by what a row and channel sum up."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1:3]
    few = Hq // Hkv * Nq <= 128
    pos = Nk - Nq + torch.arange(Nq, device="cuda")
    for b in range(B):
        o, a, x = R.attention(q[b].double(), k[b].double(), v[b].double(), pos, window, sinks, d ** -0.5)
        top = torch.nan_to_num(v[b].double(), 0, 0, 0).abs().amax((1, 2)).repeat_interleave(Hq // Hkv)[:, None, None]
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -16 if few else 2.0 ** -11) * a + (0 if few else 2.0 ** -19) * top
        tol = tol + 4 * (2.0 ** -16 * x + 2.0 ** -20) * a
        within(out[b][..., channels], o[..., channels], tol[..., channels])


WINDOWS = [  # Hq, Hkv, Nq, Nk, d, window, sinks: at most 128 rows per KV head, just above, chunks, long windows
    (4, 1, 32, 700, 64, 200, 4), (4, 1, 33, 700, 64, 200, 4), (2, 2, 128, 500, 128, 100, 70), (2, 2, 129, 500, 128, 100, 70),
    (1, 1, 700, 900, 64, 300, 0), (6, 2, 300, 2000, 128, 1500, 5), (3, 1, 400, 400, 128, 64, 0),
]


@pytest.mark.parametrize("power", [-100, -40, -20, -10, 15, 20, 60, 110])
@pytest.mark.parametrize("Hq,Hkv,Nq,Nk,d,window,sinks", WINDOWS)
def test_window_attn_values_of_any_size(Hq, Hkv, Nq, Nk, d, window, sinks, power):
    g = gen(46)
    q, k, v = rand(g, 2, Hq, Nq, d), rand(g, 2, Hkv, Nk, d), rand(g, 2, Hkv, Nk, d, std=2.0 ** power)
    v[1] = rand(g, Hkv, Nk, d)                    # the other sequence's values are of the usual size
    check_window_values(q, k, v, fbs.window_attn(q, k, v, window, sinks), window, sinks)


@pytest.mark.parametrize("Hq,Hkv,Nq,Nk,d,window,sinks", WINDOWS)
def test_window_attn_infinite_and_unseen_values(Hq, Hkv, Nq, Nk, d, window, sinks):
    """An infinity that every query sees stays in its channel and does not become a plausible number; finite values of any
    size that no query sees change no bit."""
    g = gen(47)
    q, k, v = rand(g, 1, Hq, Nq, d), rand(g, 1, Hkv, Nk, d), rand(g, 1, Hkv, Nk, d)
    good = fbs.window_attn(q, k, v, window, sinks)
    hidden = Nk - Nq - window + 1
    if hidden > sinks:
        v2 = v.clone()
        v2[:, :, sinks:hidden] = rand(g, 1, Hkv, hidden - sinks, d, std=2.0 ** 100)
        assert torch.equal(fbs.window_attn(q, k, v2, window, sinks), good)
    if sinks:
        v[:, :, sinks - 1, 5], v[:, :, sinks - 1, 7] = math.inf, math.nan
        got = fbs.window_attn(q, k, v, window, sinks)
        assert not torch.isfinite(got[..., 5]).any() and torch.isnan(got[..., 7]).all()
        rest = [c for c in range(d) if c not in (5, 7)]
        check_window_values(q, k, v, got, window, sinks, rest)


@pytest.mark.parametrize("Hq,Hkv,Nq,Nk,d,window,sinks", WINDOWS)
def test_window_attn_nan_queries(Hq, Hkv, Nq, Nk, d, window, sinks):
    """Queries of NaN, alone and all 64 of a stretch, give NaN; the others keep their bits."""
    g = gen(48)
    q, k, v = rand(g, 1, Hq, Nq, d), rand(g, 1, Hkv, Nk, d), rand(g, 1, Hkv, Nk, d)
    good = fbs.window_attn(q, k, v, window, sinks)
    bad = torch.zeros(Nq, dtype=torch.bool, device="cuda")
    bad[3] = True
    if Nq >= 256:
        bad[128:192] = True
    q[:, :, bad] = math.nan
    got = fbs.window_attn(q, k, v, window, sinks)
    assert torch.isnan(got[:, :, bad]).all() and torch.equal(got[:, :, ~bad], good[:, :, ~bad])


# ------------------------------------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (128, 0), (128, 64), (64, 16), (64, 64), (128, 128)])
def test_norm_rope_infinities_stay_where_the_formula_has_them(d, rot, interleaved):
    """An infinity makes its own channel NaN (and its pair's, where it turns) and the rest of its row 0; a NaN makes
    the row NaN; an infinite weight of a channel that does not turn reaches that channel alone."""
    g = gen(49)
    q, k = rand(g, 1, d, 5, d), rand(g, 1, 2, 5, d)
    c = torch.arange(d, device="cuda")
    q[0, c, 1, c] = math.inf                       # head i: channel i
    q[0, c, 3, c] = -math.inf
    q[0, 2, 2, 7] = math.nan
    w = torch.ones(d, device="cuda")
    if rot < d:
        w[d - 3] = math.inf
    freq = fbs.rope_freqs(rot) if rot else None
    pos = 3 + torch.arange(5, dtype=torch.int32, device="cuda")[None]
    a, _ = fbs.qk_norm_rope(q, k, freq, positions=pos, q_weight=w, interleaved=interleaved)
    ref, mag = R.norm_rope(q.double(), w, freq, pos, 1e-6, interleaved)
    assert torch.equal(torch.isnan(a), torch.isnan(ref)) and torch.equal(torch.isinf(a), torch.isinf(ref))
    fine = torch.isfinite(ref)
    within(a[fine], ref[fine], (2.0 ** -8 * ref.abs() + 2.0 ** -19 * mag)[fine])


# ------------------------------------------------------------------------------------------------------ the binding
def test_other_threads_run_while_a_call_waits_for_the_gpu():
    """With the launch queue full a call waits until the GPU has caught up; other Python threads go on meanwhile."""
    import threading
    import time
    lens, table, free = i32(3, 4), torch.zeros(2, 4, dtype=torch.int32, device="cuda"), i32(1, 2)
    slots, pos = torch.empty(2, 1, dtype=torch.int64, device="cuda"), torch.empty(2, 1, dtype=torch.int32, device="cuda")
    kv, used = torch.empty_like(lens), i32(0)
    one = torch.ones_like(lens)
    call = lambda: fbs.cache_tables(lens, one, free, table, 16, 1, slots, pos, kv, used)  # noqa: E731
    call()
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), [0.0]

    def watch():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now

    thread = threading.Thread(target=watch)
    thread.start()
    torch.cuda._sleep(1_500_000_000)                # most of a second on the GPU
    waited = 0.0
    for _ in range(20000):
        t0 = time.perf_counter()
        call()
        waited = max(waited, time.perf_counter() - t0)
        if waited > 0.1:
            break
    torch.cuda.synchronize()
    stop.set()
    thread.join()
    assert waited > 0.1, "the queue did not fill: nothing was tested"
    assert gaps[0] < 0.5 * waited


def test_outputs_too_large_for_the_gpu_raise_torchs_error():
    """1024 requests of 2^30 places (13 TB of outputs): torch's out-of-memory error, as from an allocation of its own."""
    lens = torch.zeros(1024, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        fbs.cache_tables(lens, lens, lens, torch.zeros(1024, 2, dtype=torch.int32, device="cuda"), 16, 1 << 30)


def test_kept_lengths_do_not_keep_the_slots():
    """The lengths of a step with long chunks are a tensor of their own size; where some outputs are given, only the others are
    made; small outputs share one storage of just their size."""
    R_, N = 64, 4096
    lens, new, free = (torch.zeros(R_, dtype=torch.int32, device="cuda") for _ in range(3))
    table = torch.zeros(R_, 2, dtype=torch.int32, device="cuda")
    out = fbs.cache_tables(lens, new, free, table, 64, N)
    assert [x.untyped_storage().nbytes() for x in out] == [8 * R_ * N, 4 * R_ * N, 4 * R_, 4]
    out = fbs.cache_tables(lens, new, free, table, 64, N, slots=out[0], positions=out[1])
    assert [x.untyped_storage().nbytes() for x in out[2:]] == [4 * R_ + 4] * 2
    out = fbs.cache_tables(lens, new, free, table, 64, 1)
    assert [x.untyped_storage().nbytes() for x in out] == [12 * R_ + 4 * R_ + 4] * 4
    out = fbs.cache_tables(lens[:0], new[:0], free, table[:0], 64, N, used=out[3])
    assert [tuple(x.shape) for x in out] == [(0, N), (0, N), (0,), (1,)]


# ---------------------------------------------------------------- window attention: strides, row counts, masked places
@pytest.mark.parametrize("Hq,Hkv,Nq,Nk,d,window,sinks", WINDOWS + [(1, 1, 1, 1, 64, 1, 0), (4, 1, 1, 500, 128, 64, 4), (8, 2, 1, 900, 64, 300, 0)])
def test_window_attn_strides_on_every_path(Hq, Hkv, Nq, Nk, d, window, sinks):
    """Rows in (B, N, H, d) order, with gaps between heads, tokens and sequences, 16-byte aligned only; outputs so too: the
    bits of contiguous tensors, within the tolerance that the row count sets, nothing written beside the rows."""
    g = gen(50)

    def strided(H, N):
        whole = torch.full((2, N + 3, H + 1, d + 8), 77.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole[:, 1:N + 1, :H, 8:].transpose(1, 2)

    q, k, v = rand(g, 2, Hq, Nq, d), rand(g, 2, Hkv, Nk, d), rand(g, 2, Hkv, Nk, d)
    views = []
    for x in (q, k, v):
        _, y = strided(*x.shape[1:3])
        views.append(y.copy_(x))
    whole, out = strided(Hq, Nq)
    good = fbs.window_attn(q, k, v, window, sinks)
    assert fbs.window_attn(*views, window, sinks, out=out) is out
    assert torch.equal(out, good) and torch.equal(fbs.window_attn(*views, window, sinks), good)
    check_window_values(q, k, v, good, window, sinks)
    out.fill_(77.0)
    assert (whole == 77.0).all()


@pytest.mark.parametrize("Hq,Hkv,Nq,Nk,d,window,sinks", [w for w in WINDOWS if w[3] - w[2] - w[5] + 1 > w[6] + 2] + [
    (2, 1, 200, 4000, 128, 2000, 5), (2, 1, 200, 4000, 128, 300, 5), (2, 1, 200, 4000, 64, 300, 0), (1, 1, 200, 4000, 128, 2000, 64)])
def test_window_attn_ignores_rubbish_that_no_query_sees(Hq, Hkv, Nq, Nk, d, window, sinks):
    """NaN and infinities in keys and values between the first tokens and the window, on every path: the same bits."""
    g = gen(51)
    q, k, v = rand(g, 1, Hq, Nq, d), rand(g, 1, Hkv, Nk, d), rand(g, 1, Hkv, Nk, d)
    good = fbs.window_attn(q, k, v, window, sinks)
    lo, hi = sinks, Nk - Nq - window + 1
    k[:, :, lo:hi], v[:, :, lo:hi] = math.nan, math.inf
    v[:, :, lo], v[:, :, hi - 1], k[:, :, hi - 1] = math.nan, math.nan, math.inf
    assert torch.equal(fbs.window_attn(q, k, v, window, sinks), good)


@pytest.mark.parametrize("Hq,Nq,d", SHAPES)
def test_cache_attn_nan_queries(Hq, Nq, d):
    """A query of NaN gives NaN; the others keep their bits."""
    g = gen(52)
    pool, table = filled(g, [300], 1, d, 64)
    q = rand(g, 1, Hq, Nq, d)
    good = fbs.cache4_attn(q, pool, table, i32(300))
    q[:, 1] = math.nan
    got = fbs.cache4_attn(q, pool, table, i32(300))
    keep = [h for h in range(Hq) if h != 1]
    assert torch.isnan(got[:, 1]).all() and torch.equal(got[:, keep], good[:, keep])


@pytest.mark.parametrize("Hq,Nq,d", SHAPES)
def test_cache_attn_calls_share_a_workspace_and_a_graph_replays(Hq, Nq, d):
    """Two calls one behind the other on one workspace, also captured into two graphs that share it; the workspace's old
    contents do not matter."""
    g = gen(53)
    pool, table = filled(g, [3000], 1, d, 64)
    q = rand(g, 1, Hq, Nq, d)
    kv, kv2 = i32(3000), i32(900)
    ws = torch.full((fbs.lib().sparge_cache4_attn_workspace_bytes(1, Hq, 1, Nq, d),), 255, dtype=torch.uint8, device="cuda")
    want, want2 = fbs.cache4_attn(q, pool, table, kv), fbs.cache4_attn(q, pool, table, kv2, window=100, sinks=4)
    assert torch.equal(fbs.cache4_attn(q, pool, table, kv, ws=ws), want)
    assert torch.equal(fbs.cache4_attn(q, pool, table, kv2, window=100, sinks=4, ws=ws), want2)
    s = torch.cuda.Stream()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    torch.cuda.synchronize()
    for graph, n, kw in ((graphs[0], kv, {}), (graphs[1], kv2, dict(window=100, sinks=4))):
        with torch.cuda.graph(graph, stream=s):
            outs.append(fbs.cache4_attn(q, pool, table, n, ws=ws, **kw))
    for i in (0, 1, 1, 0, 1, 0):
        ws.random_(0, 256)
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], (want, want2)[i])


@pytest.mark.parametrize("window", [830, 897, 898, 960, 1025, 1281, 1345])
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (2, 2), (4, 1)])
def test_window_attn_around_the_choice_of_kernels(Hq, Hkv, window):
    """d = 128 around the windows where the two chunk kernels take over from each other, which depends on the heads per KV head."""
    g = gen(54)
    q, k, v = rand(g, 1, Hq, 330, 128), rand(g, 1, Hkv, 1700, 128), rand(g, 1, Hkv, 1700, 128)
    check_window_values(q, k, v, fbs.window_attn(q, k, v, window, 5), window, 5)


def test_captured_window_attn_replays_on_values_of_another_size():
    """The power of two on the copy of V is found on the device: a graph captured with usual values replays on large and small
    ones, head by head."""
    g = gen(55)
    Hq, Hkv, N, d = 4, 2, 400, 64
    q, k, v = rand(g, 1, Hq, N, d), rand(g, 1, Hkv, N, d), rand(g, 1, Hkv, N, d)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    fbs.window_attn(q, k, v, 100, 3)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        out = fbs.window_attn(q, k, v, 100, 3)
    for powers in ((0, 0), (30, -30), (-50, 0), (0, 100), (0, 0)):
        for h, p in enumerate(powers):
            v[:, h] = rand(g, 1, N, d, std=2.0 ** p)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_window_values(q, k, v, out, 100, 3)
        assert torch.equal(out, fbs.window_attn(q, k, v, 100, 3))
