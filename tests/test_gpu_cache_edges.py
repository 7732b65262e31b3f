"""The cache where it can go wrong beside the ordinary: numbers that are not
finite in the part of a key that stays, how exact attention is, and queries and
scales far out."""
import math

import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs
from tests.cache_util import F64, attended, held, random_cache, tokens
from tests.test_gpu_cache import CASES, WIDE, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    mcs.last_device_status()
    yield
    assert mcs.last_device_status() == 0


@pytest.mark.parametrize("dims", [50, 18, 16])
def test_an_infinity_in_the_part_of_a_key_that_stays(dims):
    """It is held as the page's largest number; the token's other numbers, and
    every other token, are what they are without it."""
    rot = mcs.Rotary(64, dims=dims, layout="interleaved")
    g = torch.Generator().manual_seed(dims)
    K, V = (torch.randn((1, 2, 40, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    K[0, 1, 3, 60] = K[0, 0, 7, dims + 1] = 0.0                          # (so that the scales are the same)
    a, b = mcs.KVCache.empty(1, 2, 64, 64, 16), mcs.KVCache.empty(1, 2, 64, 64, 16)
    mcs.cache_append(a, K.cuda(), V.cuda(), i32(0), rotary=rot)
    K[0, 1, 3, 60], K[0, 0, 7, dims + 1] = -math.inf, math.inf
    mcs.cache_append(b, K.cuda(), V.cuda(), i32(0), rotary=rot)
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_pages.view(torch.uint8), b.v_pages.view(torch.uint8))
    (ka, _), (kb, _) = (tokens(c, 0, 40) for c in (a, b))
    top = 448 * b.k_scale[0].cpu().to(F64)
    ka[1, 3, 60], ka[0, 7, dims + 1] = -top[1], top[0]
    assert torch.equal(ka, kb)
    Q = torch.randn((1, 2, 5, 64), generator=g).to(torch.bfloat16)
    assert torch.isfinite(mcs.cache_attention(Q.cuda(), b, i32(40))).all()


def score_error(Q, cache, E, scale=None):
    """How far a row's scores may be off: E of cache_util (fp32 sums of d products), and
    for blocks of many rows the queries' two 8-bit parts, off by at most 2^-17 of
    the row's largest number each: 2^-17 max|q| sum|k| of the largest key."""
    scale = 1 / math.sqrt(Q.shape[-1]) if scale is None else scale
    keys = torch.nan_to_num(held(cache)[0].abs(), 0.0).sum(-1).max()
    return E + scale * 2.0 ** -17 * Q.to(F64).abs().amax(-1) * keys


def bound(Q, cache, lengths, A, E, scale=None):
    """How far a number may be from the definition, beside its own rounding, in
    units of the weighted magnitudes A = sum_j p_j |v_j| of its row:
    - a weight is rounded to fp16, 2^-11 of it (the sum they are divided by is not
      rounded): 2^-11;
    - a score's error moves a weight, and the sum: twice;
    - the exponential (2^-22), its argument's rounding (up to 2^7: 2^-17, twice): 2^-16;
    - fp32 sums over up to n / 16 steps of 16 keys: (n / 16) 2^-23;
    and a weight below fp16's normal range is off by 2^-25 where the row's largest
    is 2^6 or more: n of them by n 2^-31 of the row's largest term, which is at
    most n 2^-31 * max|v| (numbers and scales of these caches are alike over the pages)."""
    n = max(max(lengths), 1)
    a = 2.0 ** -11 + 2 * score_error(Q, cache, E, scale) + 2.0 ** -16 + n / 16 * 2.0 ** -23
    return a[..., None] * A + n * 2.0 ** -31 * torch.nan_to_num(held(cache)[1].abs(), 0.0).max()


def assert_within(got, ref, extra):
    got = got.cpu().to(F64)
    assert torch.isfinite(got).all()
    worst = ((got - ref).abs() / (2.0 ** -8 * ref.abs() + extra + 1e-30)).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.2f} of the bound"


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_is_as_exact_as_its_weights(case, places):
    B, Hq, H, Nq, d, page, lengths, causal, counts = CASES[case]
    cache = random_cache(B, H, lengths, d, page, seed=Nq + 1, places=places)
    g = torch.Generator().manual_seed(10)
    Q = (torch.randn((B, Hq, Nq, d), generator=g) * 1.5).to(torch.bfloat16)
    Q[..., ::3] *= 0.01
    ref, _, A, E = attended(Q, cache, lengths, causal, counts)
    O = mcs.cache_attention(Q.cuda(), cache, i32(*lengths), causal=causal, counts=None if counts is None else i32(*counts))
    assert_within(O, ref, bound(Q, cache, lengths, A, E))


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("Nq,n,d", [(1, 6, 64), (16, 6, 128), (40, 10, 64), (300, 6, 128), (300, 2, 64), (300, 400, 64)])
def test_values_that_cancel(Nq, n, d, places):
    """Neighbouring tokens with opposite values and scores close to each other:
    the output is small beside the weighted magnitudes, so the weights' own
    rounding shows (weights of 8 significant bits are off by several times the bound)."""
    B, H = 1, 8
    cache = random_cache(B, H, [n], d, 128, seed=3, spread=0.0, places=places)
    k, v = cache.k_pages.float(), cache.v_pages.float()
    k *= 2.0 ** -4
    v[:, :, 1::2] = -v[:, :, ::2]
    for to, x in ((cache.k_pages, k), (cache.v_pages, v)):
        to.view(torch.uint8).copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
    g = torch.Generator().manual_seed(10)
    Q = torch.randn((B, H, Nq, d), generator=g).to(torch.bfloat16)
    ref, _, A, E = attended(Q, cache, [n], False)
    assert (ref.abs().mean() < 0.2 * A.mean()).item()
    O = mcs.cache_attention(Q.cuda(), cache, i32(n))
    assert_within(O, ref, bound(Q, cache, [n], A, E))


@pytest.mark.parametrize("places", [0, 4096, WIDE], ids=["clusters", "idle", "dealt"])
@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("power", [-90, -60, 90, 105, 120, 127])
def test_queries_of_any_finite_size(power, Nq, places):
    """Small keys bring the scores back to an ordinary size (scales of 2^-60, and
    the softmax's scale for the rest): rows of huge and tiny numbers are as
    exact as others, where some CTAs of a cluster have no tile (idle) too."""
    d, n = 64, 200
    cache = random_cache(1, 2, [n], d, 32, seed=4, spread=0.0, places=places)
    down = min(max(-power, -60), 60)
    cache.k_scale.fill_(2.0 ** (down - 6))
    scale = 2.0 ** (-power - down - 3)
    if down - 6 < -60:
        cache.k_scale.fill_(2.0 ** -60)
        scale = 2.0 ** (60 - 6 - power - 3)
    g = torch.Generator().manual_seed(9)
    Q = torch.randn((1, 2, Nq, d), generator=g).clamp(-1.9, 1.9) * 2.0 ** power
    Q[..., ::3] *= 0.01
    Q = Q.to(torch.bfloat16)
    assert torch.isfinite(Q).all()
    ref, lse, A, E = attended(Q, cache, [n], False, scale=scale)
    O, got = mcs.cache_attention(Q.cuda(), cache, i32(n), scale=scale, return_lse=True)
    assert_within(O, ref, bound(Q, cache, [n], A, E, scale))
    assert ((got.cpu().to(F64) - lse).abs() <= score_error(Q, cache, E, scale) + 1e-5 + 1e-6 * lse.abs()).all()


@pytest.mark.parametrize("places", [0, 4096, WIDE], ids=["clusters", "idle", "dealt"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("Nq", [1, 40])
def test_scores_beyond_fp32_give_nan(Nq, sign, places):
    """All above it, all below it: NaN, and never zeros; other rows are not reached."""
    n = 200
    cache = random_cache(1, 1, [n], 64, 32, seed=4, spread=0.0, places=places)
    k = cache.k_pages.float().abs().clamp(min=1.0)
    cache.k_pages.view(torch.uint8).copy_(k.to(torch.float8_e4m3fn).view(torch.uint8))
    cache.k_scale.fill_(2.0 ** 60)
    Q = torch.full((1, 2, Nq, 64), 2.0 ** -70, dtype=torch.bfloat16, device="cuda")
    Q[0, 1] = sign * 2.0 ** 120
    for causal in (False, True):
        O, lse = mcs.cache_attention(Q, cache, i32(n), causal=causal, return_lse=True)
        assert torch.isfinite(O[0, 0]).all() and torch.isfinite(lse[0, 0]).all()
        assert O[0, 1].isnan().all() and lse[0, 1].isnan().all()


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("Nq,d,page", [(1, 64, 16), (5, 128, 64), (40, 64, 32), (300, 128, 128)])
def test_scales_of_a_callers_own(Nq, d, page, places):
    """Scales that are no powers of two; key scales of zero (scores of zero); value
    scales of zero: the page's values are zero, whatever its bytes, and its
    weights count.  (lse: the scores' error, 1e-5 and 1e-6 of it for the sum's
    rounding, log2 of a scale 2^-22 of 7: 1e-5 covers it.)"""
    lengths = [700, 300]
    cache = random_cache(2, 2, lengths, d, page, seed=8, spread=0.0, places=places)
    g = torch.Generator().manual_seed(12)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_((0.6 + torch.rand(s.shape, generator=g)).cuda())
    used = [int(p) for p in cache.page_table[cache.page_table >= 0].tolist()]
    cache.v_scale[used[0], 0] = 0.0
    cache.v_scale[used[1 % len(used)], :] = 0.0
    cache.k_scale[used[-1], 1] = 0.0
    cache.k_scale[used[0], 0] *= 4                       # (weights that would be missed)
    Q = (torch.randn((2, 4, Nq, d), generator=g) * 1.5).to(torch.bfloat16)
    for causal in (False, True):
        ref, lse, A, E = attended(Q, cache, lengths, causal)
        O, got = mcs.cache_attention(Q.cuda(), cache, i32(*lengths), causal=causal, return_lse=True)
        assert_within(O, ref, bound(Q, cache, lengths, A, E))
        got = got.cpu().to(F64)
        assert ((got - lse).abs() <= score_error(Q, cache, E) + 2e-5 + 1e-6 * lse.abs()).all()
    # all of a row's values are zero: zeros, and a finite sum
    cache.v_scale.zero_()
    O, got = mcs.cache_attention(Q.cuda(), cache, i32(*lengths), return_lse=True)
    _, lse, _, E = attended(Q, cache, lengths, False)
    assert (O == 0).all() and ((got.cpu().to(F64) - lse).abs() <= score_error(Q, cache, E) + 2e-5 + 1e-6 * lse.abs()).all()
    for x in mcs.cache_read(cache, i32(0, 0), 300)[1:]:
        assert (x == 0).all()


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -1.0, 2.0 ** 91, 2.0 ** -91])
def test_scales_out_of_range_are_recorded(bad, Nq, places):
    """A page with such a scale is left out of its head's attention, and recorded, as a bad page is."""
    cache = random_cache(1, 2, [300], 64, 32, seed=8, spread=0.0, places=places)
    g = torch.Generator().manual_seed(12)
    Q = torch.randn((1, 2, Nq, 64), generator=g).to(torch.bfloat16)
    table = cache.page_table[0].tolist()
    good_v, good_k = cache.v_scale.clone(), cache.k_scale.clone()
    ref, _, A, E = attended(Q, cache, [300], False, drop={0: list(range(64, 96))})
    other, _, A1, E1 = attended(Q, cache, [300], False)
    for t, good in ((cache.v_scale, good_v), (cache.k_scale, good_k)):
        if t is cache.k_scale and abs(bad) < 1:
            continue                                      # a small key scale is one
        t[table[2], 0] = bad
        O = mcs.cache_attention(Q.cuda(), cache, i32(300))
        assert mcs.last_device_status() == 6
        t.copy_(good)
        assert_within(O[:, 0], ref[:, 0], bound(Q, cache, [300], A, E)[:, 0])
        assert_within(O[:, 1], other[:, 1], bound(Q, cache, [300], A1, E1)[:, 1])
    assert mcs.last_device_status() == 0


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("Nq", [1, 40])
@pytest.mark.parametrize("v,k", [(-90, -6), (-75, -6), (90, -6), (-6, 90), (-6, -100)])
def test_scales_at_their_ends(v, k, Nq, places):
    """All of a head's scales far out, one page 2^20 apart: as exact as others (keys:
    the softmax's scale brings the scores back)."""
    cache = random_cache(1, 2, [300], 64, 32, seed=8, spread=0.0, places=places)
    table = cache.page_table[0].tolist()
    cache.v_scale.fill_(2.0 ** v)
    cache.v_scale[table[1]] = 2.0 ** (v - 20 if v > 0 else v + 20)
    cache.k_scale.fill_(2.0 ** k)
    scale = 2.0 ** (-9 - k)
    g = torch.Generator().manual_seed(12)
    Q = torch.randn((1, 2, Nq, 64), generator=g).to(torch.bfloat16)
    ref, lse, A, E = attended(Q, cache, [300], False, scale=scale)
    O, got = mcs.cache_attention(Q.cuda(), cache, i32(300), scale=scale, return_lse=True)
    assert_within(O, ref, bound(Q, cache, [300], A, E, scale))
    assert ((got.cpu().to(F64) - lse).abs() <= score_error(Q, cache, E, scale) + 2e-5 + 1e-6 * lse.abs()).all()


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("Nq", [1, 40, 300])
def test_far_apart_scales_are_as_exact(Nq, places):
    """Value scales 2^-26 to 2^14 over the pages, queries 2^-40 to 2^4: `bound` holds here
    too, for a row's largest term is at most the largest value, whichever page it lies in."""
    cache = random_cache(1, 2, [777], 64, 16, seed=5, spread=12.0, places=places)
    cache.k_scale.fill_(2.0 ** -7)
    g = torch.Generator().manual_seed(19)
    Q = torch.randn((1, 2, Nq, 64), generator=g) * torch.exp2(torch.randint(-40, 4, (1, 2, Nq, 1), generator=g).float())
    Q = Q.to(torch.bfloat16)
    ref, lse, A, E = attended(Q, cache, [777], False, scale=0.7)
    O, got = mcs.cache_attention(Q.cuda(), cache, i32(777), scale=0.7, return_lse=True)
    assert_within(O, ref, bound(Q, cache, [777], A, E, 0.7))
    assert ((got.cpu().to(F64) - lse).abs() <= score_error(Q, cache, E, 0.7) + 1e-5 + 1e-6 * lse.abs()).all()


@pytest.mark.parametrize("places", [64, WIDE], ids=["clusters", "dealt"])
def test_append_onto_a_page_of_zero_scales(places):
    """Tokens held at scales of 0 stand for zeros; a new token gives the page scales, and
    they stay zeros beside it."""
    cache = mcs.KVCache.empty(1, 1, places, 64, 16)
    g = torch.Generator().manual_seed(2)
    K, V = (torch.randn((1, 1, 9, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    mcs.cache_append(cache, K[:, :, :5].cuda(), V[:, :, :5].cuda(), i32(0))
    cache.k_scale.zero_()
    cache.v_scale.zero_()
    mcs.cache_append(cache, K[:, :, 5:].cuda(), V[:, :, 5:].cuda(), i32(5))
    k, v = mcs.cache_read(cache, i32(0), 9)
    assert (k[:, :, :5] == 0).all() and (v[:, :, :5] == 0).all()
    assert ((k[:, :, 5:].cpu().float() - K[:, :, 5:].float()).abs() <= K[:, :, 5:].float().abs() / 16 + 2.0 ** -15).all()
    Q = torch.randn((1, 2, 3, 64), generator=g).to(torch.bfloat16)
    ref, _, A, E = attended(Q, cache, [9], True)
    assert_within(mcs.cache_attention(Q.cuda(), cache, i32(9), causal=True), ref, bound(Q, cache, [9], A, E))
