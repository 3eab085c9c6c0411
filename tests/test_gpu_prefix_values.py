"""Attention behind a shared prefix where the tokens' weights and sizes differ by many powers of two, against fp64.

Keys are vectors of one number (a scale of 0, a minimum that bf16 holds), which f16 holds too, so a score is off by fp32 sums alone:
2^-16 of sum |q||k| scale at most, the same for all equal keys; random keys are off by half an f16 step each, which moves a score by a root
mean square of 2^-11 / sqrt 3 of |q||k| scale, less than 2^-11 here.  Values are normal numbers of both signs, so the roundings of P and of V
to f16 (half a step: 2^-11 of each) point both ways, and what they add up to has the root mean square of the outputs times at most
2^-11 each, to which the bf16 output adds at most 2^-8 / sqrt 3: less than 2^-8 in all, which the channels of all rows together are held
to, and 2^-7 those of one row (32 of them at least).  A P that is subnormal in f16 is off by 2^-25: for weights down to 2^-22 of the row's
largest that is 2^-11 of themselves again, as the largest is held at 2^8 and above."""
import pytest
import torch

import free_block_sparse_gb300 as fbs
import serving_ref as R
from test_gpu_contexts import i32, shared
from test_gpu_serving import gen

pytestmark = pytest.mark.gpu
SHARED = fbs.SPARGE_PREFIX_SHARED
# rows of a KV head in one row tile, or in two: 4 x 304 tiles of 64 tokens are 8 for each CTA, 512 tokens of a head
SETTINGS = [(2, 2, 64, 4), (2, 2, 128, 4), (70, 2, 64, 4), (70, 2, 128, 4)]  # sequences, heads of a group, d, KV heads
PREFIX, SHARE = 19456, 512


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbs.lib()
    yield
    torch.cuda.synchronize()
    assert fbs.device_status() == 0


def stored(g, B, d, H, score, v, page=64):
    """A prefix of PREFIX tokens whose keys are score[t] in every channel (or score (H, PREFIX, d)) and its values v (H, PREFIX, d); each
    sequence has one token of its own that hardly counts."""
    pool, pages, table, lens = shared(g, PREFIX, [1] * B, H, d, page)
    t = torch.arange(PREFIX, device="cuda")
    k = (score[None] if score.dim() == 3 else score[None, None, :, None].expand(1, H, PREFIX, d)).bfloat16().contiguous()
    fbs.cache4_store(k, v[None].bfloat16().contiguous(), (table[0].long()[t // page] * page + t % page)[None].contiguous(), pool)
    low = torch.full((1, H, 1, d), -60.0, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        fbs.cache4_store(low, torch.zeros_like(low), (table[b].long()[-1:] * page)[None].contiguous(), pool)
    return pool, pages, table, lens


def queries(g, B, H, G, d):
    """Rows whose sum is about d, so that a key of one number n scores about n log 2 at the scale of scale_of(d)."""
    return (1 + 0.25 * torch.randn(B, H * G, 1, d, generator=g, device="cuda")).bfloat16()


def scale_of(d):
    return 0.6931471805599453 / d


def check(q, pool, table, lens, out, d, channels, scale=None):
    """Channels (a slice) of the rows against fp64."""
    page = 16 * pool.shape[2]
    kn, ks, km, vn, vs, vm = R.read_pool(pool, d)
    K, V = R.dequantise(kn, ks, km), R.dequantise(vn, vs, vm)
    off, ref = [], []
    for b in sorted({0, 1, len(lens) // 2, len(lens) - 1}):
        n = lens[b]
        t = torch.arange(n, device="cuda")
        k, v = (x[table[b].long()[t // page], :, t % page].transpose(0, 1) for x in (K, V))
        o, _, _ = R.attention(q[b].double(), k, v, torch.tensor([n - 1], device="cuda"), 0, 0, scale or scale_of(d))
        off.append((out[b].double() - o)[..., channels].square().sum(-1))
        ref.append(o[..., channels].square().sum(-1))
    off, ref = torch.cat(off), torch.cat(ref)
    assert (ref > 0).all()
    assert off.sum() <= 2.0 ** -16 * ref.sum(), float((off.sum() / ref.sum()).sqrt())
    assert (off <= 2.0 ** -14 * ref).all(), float((off / ref).amax().sqrt())


@pytest.mark.parametrize("B,G,d,H", SETTINGS)
@pytest.mark.parametrize("at", [0, 200, 511])
@pytest.mark.parametrize("below", [6, 12, 18, 22])
def test_tokens_far_below_the_largest(B, G, d, H, at, below):
    """One token of every share takes 2^6 to 2^22 times the others' weight, but its values are zero in every second channel: there
    the others' sum is all there is."""
    g = gen(81)
    t = torch.arange(PREFIX, device="cuda")
    score = torch.where(t % SHARE == at, 0.0, -float(below))
    v = torch.randn(H, PREFIX, d, generator=g, device="cuda")
    v[:, t % SHARE == at] = (torch.arange(d, device="cuda") % 2 == 0).float()
    pool, pages, table, lens = stored(g, B, d, H, score, v)
    q = queries(g, B, H, G, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), scale=scale_of(d), path=SHARED)
    check(q, pool, table, lens, out, d, slice(1, None, 2))


@pytest.mark.parametrize("B,G,d,H", SETTINGS)
@pytest.mark.parametrize("at", [0, 200, 511])
@pytest.mark.parametrize("power", [8, 12, 16, 20, 24, 28])
def test_large_values_of_improbable_tokens(B, G, d, H, at, power):
    """A token of every share with a weight of 2^-30 of the others' has values 2^8 to 2^28 in every second channel, and zeros in the
    rest, where the others' sum stays as exact as without it."""
    g = gen(82)
    t = torch.arange(PREFIX, device="cuda")
    score = torch.where(t % SHARE == at, -30.0, 0.0)
    v = torch.randn(H, PREFIX, d, generator=g, device="cuda")
    v[:, t % SHARE == at] = (torch.arange(d, device="cuda") % 2 == 0).float() * 2.0 ** power
    pool, pages, table, lens = stored(g, B, d, H, score, v)
    q = queries(g, B, H, G, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), scale=scale_of(d), path=SHARED)
    check(q, pool, table, lens, out, d, slice(1, None, 2))


@pytest.mark.parametrize("B,G,d,H", SETTINGS)
@pytest.mark.parametrize("at", [0, 200, 511])
@pytest.mark.parametrize("power", [0, 8, 16, 30])
def test_small_values_of_a_probable_token(B, G, d, H, at, power):
    """A token of every share takes 2^12 times each other one's weight with values 2^-30 of theirs and more."""
    g = gen(83)
    t = torch.arange(PREFIX, device="cuda")
    score = torch.where(t % SHARE == at, 0.0, -12.0)
    v = torch.randn(H, PREFIX, d, generator=g, device="cuda")
    v[:, t % SHARE == at] *= 2.0 ** -power
    pool, pages, table, lens = stored(g, B, d, H, score, v)
    q = queries(g, B, H, G, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), scale=scale_of(d), path=SHARED)
    check(q, pool, table, lens, out, d, slice(None))


@pytest.mark.parametrize("B,G,d,H", SETTINGS)
@pytest.mark.parametrize("at", [0, 200, 511])
def test_zero_values(B, G, d, H, at):
    """Tokens whose values are all zero, and tiles of nothing else, beside tokens of any size."""
    g = gen(84)
    t = torch.arange(PREFIX, device="cuda")
    score = torch.where(t % SHARE == at, 0.0, -10.0)
    v = torch.randn(H, PREFIX, d, generator=g, device="cuda")
    v[:, (t % SHARE == at) | (t // 64 % 3 == 1) | (t % 5 == 0)] = 0.0
    v[:, t % 7 == 1] *= 2.0 ** 20
    pool, pages, table, lens = stored(g, B, d, H, score, v)
    q = queries(g, B, H, G, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), scale=scale_of(d), path=SHARED)
    check(q, pool, table, lens, out, d, slice(None))


@pytest.mark.parametrize("B,G,d,H", SETTINGS)
@pytest.mark.parametrize("at", [0, 200, 511])
@pytest.mark.parametrize("power", [8, 16, 24, 60, 112])
def test_large_keys_of_improbable_tokens(B, G, d, H, at, power):
    """A token of every share whose keys are 2^8 to 2^112 times the others' and point away from the queries: the others' scores stay
    as exact as without it."""
    g = gen(85)
    t = torch.arange(PREFIX, device="cuda")
    k = 2.0 * torch.randn(H, PREFIX, d, generator=g, device="cuda")
    k[:, t % SHARE == at] = -(2.0 ** power) * (0.5 + torch.rand(d, generator=g, device="cuda"))
    v = torch.randn(H, PREFIX, d, generator=g, device="cuda")
    pool, pages, table, lens = stored(g, B, d, H, k, v)
    q = queries(g, B, H, G, d)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), scale=8 * scale_of(d), path=SHARED)
    check(q, pool, table, lens, out, d, slice(None), scale=8 * scale_of(d))


@pytest.mark.parametrize("B,G,d,H", SETTINGS)
@pytest.mark.parametrize("kind", ["climbs", "falls", "peak", "turns"])
def test_scores_that_climb_and_peak(B, G, d, H, kind):
    """The references move at nearly every tile, or once, for one token late in the prefix that takes everything; a row that sees all of
    it the other way round; and what the check would say of an output that is nothing, or the values' mean."""
    g = gen(86)
    t = torch.arange(PREFIX, device="cuda")
    score = {"climbs": t * (200.0 / PREFIX), "falls": 200.0 - t * (200.0 / PREFIX), "peak": torch.where(t == 17777, 60.0, 0.0),
             "turns": t // 64 % 7 * 13.0}[kind]
    v = torch.randn(H, PREFIX, d, generator=g, device="cuda")
    pool, pages, table, lens = stored(g, B, d, H, score - 20.0, v)
    q = queries(g, B, H, G, d)
    q[1] *= -0.25                                  # (the own token's score is then +15)
    out = fbs.cache4_prefix_attn(q, pool, pages, table, i32(*lens), scale=scale_of(d), path=SHARED)
    check(q, pool, table, lens, out, d, slice(None))
    mean = v.mean(1).bfloat16()[None, :, None].expand(B, -1, G, -1).reshape(out.shape)
    for wrong in (torch.zeros_like(out), mean):
        with pytest.raises(AssertionError):
            check(q, pool, table, lens, wrong, d, slice(None))


@pytest.mark.parametrize("B", [2, 70])
@pytest.mark.parametrize("d", [64, 128])
def test_uneven_tiles_with_pages_and_numbers_that_are_not_there(B, d):
    """Tokens of any size beside pages outside the pool, and beside a value that is a NaN: the rest as without them."""
    g = gen(87)
    H, G, page = 2, 2, 16
    pool, pages, table, lens = shared(g, 1280, [1] * B, H, d, page)
    t = torch.arange(1280, device="cuda")
    size = 2.0 ** (7 * (t % 6) - 20)
    k = torch.where(t % 5 == 1, -3000.0, 1.0)[:, None] * (1 + torch.rand(H, 1280, d, generator=g, device="cuda"))
    v = torch.randn(H, 1280, d, generator=g, device="cuda") * size[:, None]
    at = (table[0].long()[t // page] * page + t % page)[None].contiguous()
    fbs.cache4_store(k[None].bfloat16().contiguous(), v[None].bfloat16().contiguous(), at, pool)
    q = queries(g, B, H, G, d)
    gone = [0, 3, 4, 5, 6, 7, 41, 79]                                       # a tile's first page, whole tiles, the last page
    kept = [j for j in range(table.shape[1]) if j not in gone]
    bad, bad_table = pages.clone(), table.clone()
    bad[gone] = torch.tensor([-1, pool.shape[0], -5, 2 ** 31 - 1, -1, -1, -1, -2 ** 31], dtype=torch.int32, device="cuda")
    bad_table[:, gone] = -1
    out = fbs.cache4_prefix_attn(q, pool, bad, bad_table, i32(*lens), scale=scale_of(d), path=SHARED)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    check(q, pool, table[:, kept].contiguous(), [n - page * len(gone) for n in lens], out, d, slice(None))
    word = 17 * d + (3 * (d // 64) + d // 64 - 1) * 4                       # token 3's word of V's last 64 channels
    pool[int(pages[20]), 0, 0, word:word + 2] = 255
    got = fbs.cache4_prefix_attn(q, pool, bad, bad_table, i32(*lens), scale=scale_of(d), path=SHARED)
    assert fbs.device_status() == fbs.SPARGE_ERR_INVALID_ARG
    assert torch.isnan(got[:, :G, :, d - 64:]).all() and torch.equal(got[:, G:], out[:, G:])
    if d == 128:                                                           # (the token's other channels, under another power)
        off = (got[:, :G, :, :64].double() - out[:, :G, :, :64].double()).square().sum()
        assert off <= 2.0 ** -14 * out[:, :G, :, :64].double().square().sum()
