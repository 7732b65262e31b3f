"""The 8-bit cache against definitions in 64 bits: appending (scales, earlier
tokens moved to a larger one, rotation, ragged counts, numbers that are not
finite), reading back, and attention over it."""
import math

import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs
from tests.cache_util import (F64, assert_attention, attended, held, nearest_e4m3, random_cache, scale_for, tokens, turned)

pytestmark = pytest.mark.gpu

# room for more than 64 tiles of 128 tokens: the work is dealt over all SMs, and
# more than 16 rows of a key head take the tensor-memory kernel
WIDE = 8320


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def clean_status():
    mcs.last_device_status()
    yield
    assert mcs.last_device_status() == 0


class HostCache:
    """What append does, token by token on the host in 64 bits: numbers and scales of every page."""

    def __init__(self, cache):
        self.page, self.table = cache.page, cache.page_table.cpu().tolist()
        self.x = [t.cpu().float().to(F64) for t in (cache.k_pages, cache.v_pages)]
        self.s = [t.cpu().to(F64) for t in (cache.k_scale, cache.v_scale)]

    def append(self, K, V, start, counts):
        for b in range(K.shape[0]):
            at, end = start[b], start[b] + counts[b]
            if counts[b] == 0:
                continue
            for p in range(at // self.page, -(-end // self.page)):
                lo, hi = max(at, p * self.page), min(end, (p + 1) * self.page)
                pid, slot, n_old = self.table[b][p], lo - p * self.page, max(0, at - p * self.page)
                for h in range(K.shape[1]):
                    for w, src in enumerate((K, V)):
                        new = src[b, h, lo - at:hi - at]
                        s = scale_for(new.abs().max().item())
                        if n_old:
                            s = max(s, self.s[w][pid, h].item())
                            self.x[w][pid, h, :n_old] = nearest_e4m3(self.x[w][pid, h, :n_old] * (self.s[w][pid, h] / s))
                        self.s[w][pid, h] = s
                        self.x[w][pid, h, slot:slot + hi - lo] = nearest_e4m3((new / s).clamp(-448, 448))


def same_cache(cache, host, rotated_keys=False):
    for w, (pages, scale) in enumerate(((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale))):
        got, s = pages.cpu().float().to(F64), scale.cpu().to(F64)
        if rotated_keys and w == 0:
            # fp32 rotation moves a number by 5e-7 of the largest at most: next to a border between two e4m3 numbers
            # it takes the other one, a step of at most 2^-3 of it away (2^-9 * scale below the normal range)
            a, r = got * s[..., None, None], host.x[w] * host.s[w][..., None, None]
            off = (a - r).abs()
            assert (off <= 2.0 ** -3 * r.abs() + 2.0 ** -9 * s[..., None, None] + 1e-6 * r.abs().max()).all()
            assert (off > 1e-6 * r.abs().max()).double().mean() < 1e-3
        else:
            assert torch.equal(s, host.s[w])
            assert torch.equal(got, host.x[w])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_append_and_read(page, d):
    """Calls of many sizes one after another, pages that end inside a call, a
    call that grows the scale of what is held, ragged counts: every byte."""
    B, H = 3, 2
    cache = mcs.KVCache.empty(B, H, 5 * 128, d, page)
    host = HostCache(cache)
    g = torch.Generator().manual_seed(page + d)
    at = [0, 0, 0]
    for i, n in enumerate([1, 1, 15, 3, 64, 1, 129, 200, 2]):
        size = [1.0, 30.0, 1e-3, 1.0, 1e4, 1.0, 0.1, 3.0, 1e-20][i]
        K = (torch.randn((B, n, H, d), generator=g) * size).to(torch.bfloat16).transpose(1, 2)
        V = (torch.randn((B, H, n, d), generator=g) / size).to(torch.bfloat16)
        counts = [n, n // 2, max(0, n - 1)] if i % 3 == 2 else [n] * 3
        mcs.cache_append(cache, K.cuda().contiguous().transpose(1, 2).contiguous().transpose(1, 2) if i % 2 else K.cuda(), V.cuda(),
                         i32(*at), counts=i32(*counts) if i % 3 == 2 else None)
        host.append(K.to(F64), V.to(F64), at, counts)
        at = [a + c for a, c in zip(at, counts)]
        # sequences must not share a place, so the host and the device agree on everything
        same_cache(cache, host)
    n = max(at) + 5
    start = i32(0, 3, 0)
    K, V = mcs.cache_read(cache, start, n, counts=i32(n, n - 7, 0))
    k, v = held(cache)
    for b, (s, c) in enumerate(((0, n), (3, n - 7), (0, 0))):
        kk, vv = tokens(cache, b, s + c)
        for got, ref in ((K[b], kk), (V[b], vv)):
            assert torch.equal(got[:, :c].cpu().to(F64), ref[:, s:].to(torch.bfloat16).to(F64))
            assert (got[:, c:] == 0).all()


def test_append_overwrites_and_starts_pages_afresh():
    """A call sets the sequence's end: a page begun anew takes a scale of its own, whatever it held."""
    cache = mcs.KVCache.empty(1, 1, 64, 64, 16)
    host = HostCache(cache)
    g = torch.Generator().manual_seed(1)
    for at, n, size in ((0, 40, 1e3), (16, 10, 1e-3), (20, 30, 1.0), (0, 3, 1e-6)):
        K, V = ((torch.randn((1, 1, n, 64), generator=g) * size).to(torch.bfloat16) for _ in range(2))
        mcs.cache_append(cache, K.cuda(), V.cuda(), i32(at))
        host.append(K.to(F64), V.to(F64), [at], [n])
        same_cache(cache, host)


@pytest.mark.parametrize("layout,d,dims,axes", [("half", 128, 128, None), ("interleaved", 64, 50, None), ("half", 64, 48, (8, 8, 8))])
def test_append_rotates_keys(layout, d, dims, axes):
    B, H, n = 2, 3, 77
    rot = mcs.Rotary(d, dims=dims, layout=layout, axes=axes)
    cache = mcs.KVCache.empty(B, H, 300, d, 32)
    host = HostCache(cache)
    g = torch.Generator().manual_seed(5)
    at = [5, 130]
    first = [torch.randn((B, H, 130, d), generator=g).to(torch.bfloat16) for _ in range(2)]
    mcs.cache_append(cache, first[0].cuda(), first[1].cuda(), i32(0, 0), counts=i32(*at))
    host.append(first[0].to(F64), first[1].to(F64), [0, 0], at)
    K, V = (torch.randn((B, H, n, d), generator=g).to(torch.bfloat16) for _ in range(2))
    if axes:
        pos = torch.randint(0, 1000, (B, n, 3), generator=g, dtype=torch.int32)
        mcs.cache_append(cache, K.cuda(), V.cuda(), i32(*at), rotary=rot, positions=pos.cuda())
    else:
        pos = (torch.tensor(at)[:, None] + torch.arange(n)).to(torch.int32)[..., None]
        mcs.cache_append(cache, K.cuda(), V.cuda(), i32(*at), rotary=rot)
    host.append(turned(K, pos, rot), V.to(F64), at, [n, n])
    same_cache(cache, host, rotated_keys=True)


@pytest.mark.parametrize("places", [64, WIDE], ids=["clusters", "dealt"])
def test_numbers_that_are_not_finite(places):
    """+-inf is held as the page's largest number, a token with a NaN as a NaN
    key: rows that see it are NaN, rows that do not are not reached."""
    cache = mcs.KVCache.empty(1, 1, places, 64, 32)
    g = torch.Generator().manual_seed(2)
    K, V = (torch.randn((1, 1, 40, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    K[0, 0, 3, 7], V[0, 0, 5, 1] = math.inf, -math.inf
    K[0, 0, 30, 2], V[0, 0, 33, 9] = math.nan, math.nan
    mcs.cache_append(cache, K.cuda(), V.cuda(), i32(0))
    k, v = tokens(cache, 0, 40)
    s = cache.k_scale.cpu().to(F64)[:, 0], cache.v_scale.cpu().to(F64)[:, 0]
    assert k[0, 3, 7] == 448 * s[0][0] and v[0, 5, 1] == -448 * s[1][0]
    assert s[0][0] <= 4 / 224 and s[1][0] <= 5 / 224                  # inf does not set the scale
    bad = k[0].isnan()
    assert bad[30].all() and bad[33].all() and bad.sum() == 128
    assert not v.isnan().any() and v[0, 33, 9] == 0
    Q = torch.randn((1, 1, 40, 64), generator=g).to(torch.bfloat16).cuda()
    O = mcs.cache_attention(Q, cache, i32(40), causal=True)
    assert torch.isfinite(O[0, 0, :30]).all() and O[0, 0, 30:].isnan().all()
    assert mcs.cache_attention(Q, cache, i32(40)).isnan().all()
    assert torch.isfinite(mcs.cache_attention(Q, cache, i32(30))).all()
    # a query that is not finite gives NaN, and no other row
    Q[0, 0, 4, 0], Q[0, 0, 9, 0] = math.nan, math.inf
    for rows in (40, 10):
        O = mcs.cache_attention(Q[:, :, :rows].contiguous(), cache, i32(30))
        fine = torch.ones(rows, dtype=torch.bool)
        fine[[4, 9]] = False
        assert torch.isfinite(O[0, 0, fine.cuda()]).all() and O[0, 0, [4, 9]].isnan().all()


CASES = [
    # B, Hq, H, Nq, d, page, lengths, causal, counts
    (1, 1, 1, 1, 64, 16, [1], True, None),
    (1, 4, 4, 1, 128, 64, [333], False, None),
    (3, 8, 2, 1, 128, 16, [1, 130, 4097], True, None),
    (4, 4, 4, 1, 64, 128, [0, 127, 128, 129], False, None),
    (2, 12, 4, 5, 64, 32, [3, 900], True, None),
    (2, 12, 4, 5, 128, 32, [700, 31], True, [5, 2]),
    (3, 2, 1, 9, 128, 64, [65, 0, 640], False, [9, 9, 0]),
    (1, 2, 2, 17, 64, 16, [15], True, None),
    (1, 6, 3, 33, 128, 128, [515], True, None),
    (2, 2, 2, 130, 64, 64, [140, 77], True, None),
    (1, 1, 1, 257, 128, 64, [1000], False, None),
    (2, 8, 2, 70, 128, 16, [257, 2049], True, [70, 64]),
    (1, 3, 1, 300, 64, 32, [300], True, None),
    (2, 2, 1, 512, 128, 128, [129, 1537], True, [512, 400]),
    (1, 5, 5, 256, 64, 64, [128], False, None),
    (1, 4, 1, 700, 128, 32, [11], True, None),
    # enough places for the work to be dealt over all SMs: lengths far apart, parts that end anywhere
    (5, 4, 2, 1, 64, 16, [8300, 1, 0, 700, 4097], True, None),
    (1, 3, 1, 1, 128, 128, [20001], False, None),
    (2, 4, 2, 10, 128, 32, [8193, 8200], True, [10, 3]),
    (9, 2, 2, 1, 64, 64, [9000, 0, 0, 130, 129, 128, 127, 1, 8000], False, None),
    (40, 8, 8, 1, 64, 16, [(37 * i * i) % 700 for i in range(40)], True, None),
    (2, 2, 1, 300, 64, 16, [8400, 299], True, [300, 299]),
    (1, 3, 3, 400, 128, 64, [400], True, None),
]


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(case, places):
    B, Hq, H, Nq, d, page, lengths, causal, counts = case
    cache = random_cache(B, H, lengths, d, page, seed=Nq, places=places)
    g = torch.Generator().manual_seed(9)
    Q = (torch.randn((B, Hq, Nq, d), generator=g) * 1.5).to(torch.bfloat16)
    Q[..., :: 3] *= 0.01
    ref, lse, A, E = attended(Q, cache, lengths, causal, counts)
    O, got_lse = mcs.cache_attention(Q.cuda(), cache, i32(*lengths), causal=causal, return_lse=True,
                                     counts=None if counts is None else i32(*counts))
    assert_attention(O, ref, A, E, weight=2.0 ** -11 if Nq * Hq // H <= 16 else 2.0 ** -8)
    got_lse = got_lse.cpu().to(F64)
    assert torch.equal(got_lse.isinf(), lse.isinf())
    some = ~lse.isinf()
    assert ((got_lse - lse).abs()[some] <= (2 * E + 1e-5 + 1e-6 * lse.abs())[some]).all()
    again = mcs.cache_attention(Q.cuda(), cache, i32(*lengths), causal=causal,
                                counts=None if counts is None else i32(*counts))
    assert torch.equal(O, again)


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
@pytest.mark.parametrize("Nq", [1, 40, 300])
@pytest.mark.parametrize("spread", [0.0, 12.0])
def test_attention_with_far_apart_scales_and_sharp_scores(Nq, spread, places):
    """Pages whose scales differ by many binades (a row's largest score need not
    carry its largest weight), large and tiny queries, another softmax scale."""
    lengths = [777]
    cache = random_cache(1, 2, lengths, 64, 16, seed=4, spread=spread, places=places)
    cache.k_scale.fill_(2.0 ** -7)
    g = torch.Generator().manual_seed(9)
    Q = (torch.randn((1, 2, Nq, 64), generator=g) * torch.exp2(torch.randint(-40, 4, (1, 2, Nq, 1), generator=g).float())).to(torch.bfloat16)
    ref, lse, A, E = attended(Q, cache, lengths, False, scale=0.7)
    O = mcs.cache_attention(Q.cuda(), cache, i32(777), scale=0.7)
    # 2^-25 of the largest weight for those below fp16's normal range: 777 of them at most, on the largest numbers
    assert_attention(O, ref, A, E, weight=2.0 ** -11 if Nq <= 16 else 2.0 ** -8)


@pytest.mark.parametrize("places", [0, WIDE], ids=["clusters", "dealt"])
def test_bad_pages_and_lengths_are_left_out_and_recorded(places):
    lengths = [200, 64]
    cache = random_cache(2, 1, lengths, 64, 32, seed=6, places=places)
    cache.page_table[0, 2] = -7                       # places 64..95 of sequence 0
    cache.page_table[0, 5] = cache.n_pages            # places 160..191
    g = torch.Generator().manual_seed(9)
    for Nq in (1, 200):
        Q = torch.randn((2, 2, Nq, 64), generator=g).to(torch.bfloat16)
        keep = cache.page_table.clone()
        cache.page_table[0, 2] = cache.page_table[0, 5] = int(keep[0, 0])
        ref, _, A, E = attended(Q, cache, lengths, False, drop={0: list(range(64, 96)) + list(range(160, 192))})
        cache.page_table.copy_(keep)
        O = mcs.cache_attention(Q.cuda(), cache, i32(*lengths))
        assert mcs.last_device_status() == 6
        assert_attention(O, ref, A, E, weight=2.0 ** -8)
    cap = cache.capacity
    K, V = mcs.cache_read(cache, i32(60, cap - 3), 8)
    assert mcs.last_device_status() == 6
    assert (K[0, :, 4:] == 0).all() and (K[1, :, 3:] == 0).all()
    before = [t.view(torch.uint8).clone() for t in (cache.k_pages, cache.v_pages)]
    new = torch.ones((2, 1, 40, 64), dtype=torch.bfloat16, device="cuda")
    mcs.cache_append(cache, new, new, i32(64, -1), counts=i32(32, 40))
    assert mcs.last_device_status() == 6
    mcs.cache_append(cache, new, new, i32(cap, cap), counts=i32(40, 0))
    assert mcs.last_device_status() == 6
    assert torch.equal(before[0], cache.k_pages.view(torch.uint8)) and torch.equal(before[1], cache.v_pages.view(torch.uint8))
    # lengths beyond the table's places count as those
    full = random_cache(1, 1, [96], 64, 32, seed=8)
    short = mcs.KVCache(full.k_pages, full.v_pages, full.k_scale, full.v_scale,
                        torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"))
    short.k_pages.view(torch.uint8).bitwise_and_(0xBF)
    short.v_pages.view(torch.uint8).bitwise_and_(0xBF)
    Q = torch.randn((1, 1, 1, 64), generator=g).to(torch.bfloat16).cuda()
    a = mcs.cache_attention(Q, short, i32(5000))
    assert mcs.last_device_status() == 6
    assert torch.equal(a, mcs.cache_attention(Q, short, i32(64)))


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes, its last pages in use."""
    H, page, d = 2, 128, 128
    n_pages = 2 ** 32 // (H * page * d) + 40
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB")
    pools = [torch.empty((n_pages, H, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((n_pages, H), device="cuda") for _ in range(2)]
    table = torch.tensor([[n_pages - 1, 3, n_pages - 5, n_pages - 2]], dtype=torch.int32, device="cuda")
    big = mcs.KVCache(*[p.view(torch.float8_e4m3fn) for p in pools], *scales, table)
    small = mcs.KVCache.empty(1, H, 4 * page, d, page)
    g = torch.Generator(device="cuda").manual_seed(2)
    K, V = (torch.randn((1, H, 500, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for c in (big, small):
        mcs.cache_append(c, K, V, i32(0))
    for a, b in zip(mcs.cache_read(big, i32(0), 500), mcs.cache_read(small, i32(0), 500)):
        assert torch.equal(a, b)
    for Nq in (1, 300):
        Q = torch.randn((1, H, Nq, d), generator=g, device="cuda").to(torch.bfloat16)
        assert torch.equal(mcs.cache_attention(Q, big, i32(500), causal=True), mcs.cache_attention(Q, small, i32(500), causal=True))


def test_graphs_that_share_a_cache_and_streams():
    """Two captured generation steps over one cache, replayed in turn, and an
    eager call on another stream at the same time: places and lengths live on
    the device, and no call leaves anything behind for the next."""
    cache = random_cache(2, 2, [100, 300], 128, 32, seed=3, poison=False)
    lengths = i32(100, 300)
    g = torch.Generator(device="cuda").manual_seed(4)
    Qs = [torch.randn((2, 4, n, 128), generator=g, device="cuda").to(torch.bfloat16) for n in (1, 150)]
    outs = [torch.empty_like(q) for q in Qs]
    for q, o in zip(Qs, outs):
        mcs.cache_attention(q, cache, lengths, causal=True, out=o)
    torch.cuda.synchronize()
    graphs = []
    for q, o in zip(Qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mcs.cache_attention(q, cache, lengths, causal=True, out=o)
        graphs.append(graph)
    for step in range(3):
        for q in Qs:
            q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        lengths.sub_(step)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(side):
            eager = [mcs.cache_attention(q, cache, lengths, causal=True) for q in Qs]
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e)


def test_lengths_and_counts_out_of_range():
    """Negative ones count as none, counts above the call's rows as all of them."""
    for places in (0, WIDE):
        cache = random_cache(2, 1, [50, 70], 64, 16, seed=1, places=places, poison=False)
        g = torch.Generator().manual_seed(3)
        Q = torch.randn((2, 4, 9, 64), generator=g).to(torch.bfloat16).cuda()
        O = mcs.cache_attention(Q, cache, i32(-3, 70), counts=i32(9, -1))
        assert (O == 0).all()
        assert torch.equal(mcs.cache_attention(Q, cache, i32(50, 70), causal=True, counts=i32(2 ** 31 - 1, 9)),
                           mcs.cache_attention(Q, cache, i32(50, 70), causal=True))
        K, V = mcs.cache_read(cache, i32(0, 0), 5, counts=i32(-1, 99))
        assert (K[0] == 0).all() and (V[0] == 0).all() and (K[1] != 0).any()


@pytest.mark.parametrize("capacity", [400, WIDE], ids=["clusters", "dealt"])
def test_generation_loop(capacity):
    """The operators together, as a generating model uses them: chunks and then
    single tokens, each rotated, appended and attended with everything before;
    against attention in 64 bits over what the cache holds, and the context
    read back for a dense call."""
    B, Hq, H, d, page = 2, 6, 2, 64, 16
    rot = mcs.Rotary(d, scaling=("ntk", 2.0))
    cache = mcs.KVCache.empty(B, H, capacity, d, page)
    host = HostCache(cache)
    g = torch.Generator().manual_seed(11)
    at = [0, 0]
    for n in (100, 37, 1, 1, 150, 1):
        qkv = torch.randn((B, n, Hq + 2 * H, d), generator=g).to(torch.bfloat16).cuda()
        q, k, v = (t.transpose(1, 2) for t in qkv.split((Hq, H, H), 2))
        start = i32(*at)
        pos = start[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")
        Q = mcs.rotate(q, pos, rot)
        mcs.cache_append(cache, k, v, start, rotary=rot)
        host.append(turned(k, pos[..., None], rot), v.cpu().to(F64), at, [n, n])
        same_cache(cache, host, rotated_keys=True)
        host = HostCache(cache)                       # go on from what the cache holds
        at = [a + n for a in at]
        O = mcs.cache_attention(Q, cache, i32(*at), causal=True)
        ref, _, A, E = attended(Q, cache, at, True)
        assert_attention(O, ref, A, E, weight=2.0 ** -8)
    K, V = mcs.cache_read(cache, i32(0, 0), at[0])
    Q = torch.randn((B, H, at[0], d), generator=g).to(torch.bfloat16).cuda()
    D = mcs.dense(Q, K, V)
    O = mcs.cache_attention(Q, cache, i32(*at))
    ref, _, A, E = attended(Q, cache, at, False)
    assert_attention(O, ref, A, E, weight=2.0 ** -8)
    assert_attention(D, ref, A, E, weight=2.0 ** -8)
