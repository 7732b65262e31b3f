"""Definitions in 64 bits of the rotary and cache operators, token by token on
the host, and the bounds their outputs are held to."""
import math

import torch

from sparse_attention_diffusion_mcs_b200 import KVCache

F64 = torch.float64


def turned(x, pos, rotary, back=False):
    """x [B, H, N, d], pos [B, N, axes]: the rotation in 64 bits, from the rotary's own description."""
    x = x.detach().to(F64).cpu().clone()
    pos = pos.cpu().to(F64)
    p = rotary.dims // 2
    axis = [a for a, m in enumerate(rotary.axes) for _ in range(m)]
    for i in range(p):
        j, k = (i, p + i) if rotary.layout == "half" else (2 * i, 2 * i + 1)
        t = (pos[..., axis[i]] * rotary.frequencies[i])[:, None]
        c, s = torch.cos(t) * rotary.magnitude, torch.sin(t) * rotary.magnitude
        if back:
            s = -s
        a, b = x[..., j].clone(), x[..., k].clone()
        x[..., j], x[..., k] = a * c - b * s, a * s + b * c
    return x


def nearest_e4m3(x):
    """Nearest e4m3 number (ties to even) of 64-bit x, |x| <= 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).to(F64) - 3)
    return torch.round(x / step) * step


def scale_for(amax):
    """The smallest 2^e, |e| <= 60, with amax <= 448 * 2^e."""
    e = -60
    while e < 60 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def held(cache):
    """(K, V) float64 [n_pages, H, page, d] that the cache's numbers stand for."""
    k = cache.k_pages.cpu().to(torch.float32).to(F64) * cache.k_scale.cpu().to(F64)[..., None, None]
    v = cache.v_pages.cpu().to(torch.float32).to(F64) * cache.v_scale.cpu().to(F64)[..., None, None]
    return k, v


def random_cache(B, H, lengths, d, page, seed=0, spread=1.0, spare=3, poison=True, places=0):
    """A cache whose sequences hold `lengths` tokens in pages dealt out of
    order; what no token owns (tails of last pages, spare pages) is NaN, and
    table entries behind the last page are -1.  places: the table has room for
    as many tokens at least (what decides how the work is dealt)."""
    g = torch.Generator().manual_seed(seed)
    per = max(max(1, max(-(-n // page) for n in lengths)) + 1, places // page)
    need = sum(-(-n // page) for n in lengths)
    n_pages = need + spare
    pages, scales = [], []
    for _ in range(2):
        x = torch.randn((n_pages, H, page, d), generator=g) * 60
        pages.append(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        e = torch.round(torch.randn((n_pages, H), generator=g) * spread).clamp(-20, 20)
        scales.append(torch.exp2(e - 6.0))
    table = torch.full((B, per), -1, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=g)[:need].tolist()
    own = torch.zeros((n_pages, page), dtype=torch.bool)
    for b, n in enumerate(lengths):
        for i in range(-(-n // page)):
            table[b, i] = order.pop()
            own[table[b, i], :min(page, n - i * page)] = True
    if poison:
        for x in pages:
            x[~own[:, None, :, None].expand_as(x)] = 0x7F
    return KVCache(*[x.cuda().view(torch.float8_e4m3fn) for x in pages], *[s.cuda() for s in scales], table.cuda())


def tokens(cache, b, n):
    """(K, V) float64 [H, n, d] of the first n tokens of sequence b."""
    k, v = held(cache)
    table = cache.page_table[b].cpu().tolist()
    at = [(table[j // cache.page], j % cache.page) for j in range(n)]
    if n == 0:
        z = torch.zeros((cache.H, 0, cache.d), dtype=F64)
        return z, z
    p, s = torch.tensor([a for a, _ in at]), torch.tensor([a for _, a in at])
    return k[p, :, s].transpose(0, 1), v[p, :, s].transpose(0, 1)


def attended(Q, cache, lengths, causal, counts=None, scale=None, drop=None):
    """(O, lse, A, E) in 64 bits: the output, the log sum of exp, the weighted
    mean magnitude sum_j p_ij |v_j| of each output number, and a bound on a
    score's rounding in each row.  drop[b]: places left out."""
    B, Hq, Nq, d = Q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    O = torch.zeros((B, Hq, Nq, d), dtype=F64)
    A, L, E = torch.zeros_like(O), torch.full((B, Hq, Nq), -math.inf, dtype=F64), torch.zeros((B, Hq, Nq), dtype=F64)
    q64 = Q.cpu().to(F64)
    for b in range(B):
        n = lengths[b]
        nq = Nq if counts is None else max(0, min(counts[b], Nq))
        k, v = tokens(cache, b, n)
        for h in range(Hq):
            kk, vv = k[h * cache.H // Hq], v[h * cache.H // Hq]
            s = scale * q64[b, h] @ kk.T
            see = torch.ones((Nq, n), dtype=torch.bool)
            if causal:
                see = torch.arange(n)[None] <= (n - nq + torch.arange(Nq))[:, None]
            see[nq:] = False
            for j in (drop or {}).get(b, ()):
                see[:, j] = False
            s = torch.where(see, s, -math.inf)
            m = s.amax(-1, keepdim=True) if n else torch.full((Nq, 1), -math.inf, dtype=F64)
            p = torch.where(see, torch.exp(s - torch.where(m.isinf(), 0.0, m)), 0.0)
            tot = p.sum(-1, keepdim=True)
            some = (tot > 0).expand(-1, d)
            w = p / torch.where(tot > 0, tot, 1.0)
            vz = torch.where(see.any(0)[:, None], vv, 0.0)
            O[b, h] = torch.where(some, w @ vz, 0.0)
            A[b, h] = torch.where(some, w @ vz.abs(), 0.0)
            L[b, h] = (m + torch.log(tot))[:, 0]
            kz = torch.where(see.any(0)[:, None], kk, 0.0)
            # fp32 accumulation of d exact products, the query's fp16 form (2^-25 of its largest number), the
            # factors' roundings: (d + 4) 2^-24 sum |q||k|, at most
            E[b, h] = scale * (d + 4) * 2.0 ** -24 * (q64[b, h].abs() @ kz.abs().T).amax(-1) if n else 0.0
    return O, L, A, E


def assert_attention(got, ref, A, E, weight=2.0 ** -11):
    """got bf16 against ref: half a step of bf16 (2^-8), and the weights' own
    rounding (`weight`), a score's (E, once in the weight and once in the sum)
    and the exponential's (2^-22 and, of its argument up to 2^7, 2^-17) on the
    weighted magnitudes; a weight below fp16's normal range is off by 2^-25 of
    the largest: over a row of n of them, at most 2^-11 of the magnitudes where
    n <= 2^14."""
    got = got.cpu().to(F64)
    assert torch.isfinite(got).all()
    tol = 2.0 ** -8 * ref.abs() + (2 * weight + 2.0 ** -16 + 2 * E[..., None]) * A + 1e-30
    worst = ((got - ref).abs() / tol).max().item() if ref.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.2f} of the bound"
