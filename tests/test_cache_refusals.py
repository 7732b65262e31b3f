"""What the rotary and cache entry points refuse: the C functions before any
launch (no GPU needed), and the Python calls on shapes, types, layouts and
devices that the library would read or write wrongly."""
import ctypes

import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs
from sparse_attention_diffusion_mcs_b200 import _lib
from sparse_attention_diffusion_mcs_b200 import build as _build
from sparse_attention_diffusion_mcs_b200.rotary import _position_strides

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000
I64x3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def L():
    _build.build()
    return _lib.lib()


def rotary(**kw):
    v = dict(dict(turns=FAKE, axis=FAKE, pairs=32, interleaved=0, axes=1, magnitude=1.0), **kw)
    return ctypes.byref(_lib.McsRotary(*v.values()))


def cache(**kw):
    v = dict(dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, n_pages=8, max_pages=4, B=2, H=2, page=16, d=64), **kw)
    return ctypes.byref(_lib.McsCache(*v.values()))


def test_rotate(L):
    def call(rot=rotary(), **kw):
        v = dict(dict(x=FAKE, dtype=0, B=1, H=2, N=3, d=64, strides=I64x3(384, 64, 128), pos=FAKE, pb=0, pn=1), **kw)
        return L.mcs_rotate(v["x"], v["dtype"], v["B"], v["H"], v["N"], v["d"], v["strides"], v["pos"], v["pb"], v["pn"],
                            rot, 0, v.get("out", FAKE), None)
    for B, H, N in ((0, 2, 3), (1, 0, 3), (1, 2, 0)):
        assert call(B=B, H=H, N=N) == OK
    assert call(dtype=3) == UNSUPPORTED
    assert call(rot=None) == INVALID
    for bad in (dict(pairs=33), dict(pairs=-1), dict(axes=0), dict(magnitude=0.0), dict(magnitude=float("inf")),
                dict(turns=0), dict(axis=0), dict(turns=FAKE + 4)):
        assert call(rot=rotary(**bad)) == INVALID
    for bad in (dict(x=0), dict(out=0), dict(pos=0), dict(pos=FAKE + 2), dict(B=-1), dict(d=0), dict(x=FAKE + 1),
                dict(dtype=2, x=FAKE + 2), dict(B=2 ** 30, N=4)):
        assert call(**bad) == INVALID


CACHES = [(dict(k=0), INVALID), (dict(table=0), INVALID), (dict(v=FAKE + 8), INVALID), (dict(ks=FAKE + 2), INVALID),
          (dict(d=96), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(B=0), INVALID), (dict(n_pages=0), INVALID),
          (dict(max_pages=0), INVALID), (dict(B=32768, H=2), INVALID), (dict(max_pages=2 ** 27), INVALID),
          (dict(n_pages=2 ** 27), INVALID)]


@pytest.mark.parametrize("bad,code", CACHES)
def test_a_cache_that_is_none(L, bad, code):
    c = cache(**bad)
    s = I64x3(0, 0, 64)
    assert L.mcs_cache_append(c, FAKE, FAKE, s, s, 1, FAKE, None, None, 0, 0, None, None) == code
    assert L.mcs_cache_read(c, FAKE, None, 1, FAKE, FAKE, None) == code
    assert L.mcs_cache_attention(c, FAKE, 2, 1, FAKE, None, 0, 0.125, FAKE, None, FAKE, 2 ** 30, None) == code
    assert L.mcs_cache_attention_workspace_size(c, 2, 1) == 0


def test_append_read_attention(L):
    c = cache()

    def append(**kw):
        v = dict(dict(K=FAKE, V=FAKE, ks=I64x3(128, 64, 128), vs=I64x3(128, 64, 128), n=2, start=FAKE, counts=None, pos=None,
                      rot=None), **kw)
        return L.mcs_cache_append(c, v["K"], v["V"], v["ks"], v["vs"], v["n"], v["start"], v["counts"], v["pos"], 0, 1,
                                  v["rot"], None)
    assert append(n=0) == OK
    assert append(rot=rotary(pairs=12)) == UNSUPPORTED                   # half layout: whole vectors
    for bad in (dict(K=0), dict(V=0), dict(start=None), dict(n=-1), dict(K=FAKE + 2), dict(counts=FAKE + 2),
                dict(ks=I64x3(128, 60, 128)), dict(vs=I64x3(128, 64, 127)), dict(rot=rotary(axes=3)),
                dict(rot=rotary(pairs=40)), dict(ks=None), dict(n=2 ** 30 + 1)):
        assert append(**bad) == INVALID

    assert L.mcs_cache_read(c, FAKE, None, 0, FAKE, FAKE, None) == OK
    for bad in ((None, None, 1, FAKE, FAKE), (FAKE, FAKE + 1, 1, FAKE, FAKE), (FAKE, None, -1, FAKE, FAKE),
                (FAKE, None, 1, FAKE + 2, FAKE), (FAKE, None, 1, FAKE, None)):
        assert L.mcs_cache_read(c, *bad, None) == INVALID

    def attend(Q=FAKE, Hq=4, Nq=1, lengths=FAKE, counts=None, scale=0.125, O=FAKE, lse=None, ws=FAKE):
        return L.mcs_cache_attention(c, Q, Hq, Nq, lengths, counts, 0, scale, O, lse, ws, 2 ** 30, None)
    assert attend(Nq=0) == OK
    for bad in (dict(Q=None), dict(O=None), dict(lengths=None), dict(Hq=3), dict(Hq=0), dict(Nq=-1), dict(scale=0.0),
                dict(scale=float("nan")), dict(Q=FAKE + 8), dict(counts=FAKE + 2), dict(lse=FAKE + 1),
                dict(ws=FAKE + 8), dict(Nq=2 ** 20, Hq=4)):
        assert attend(**bad) == INVALID


def test_a_rotary_that_is_none():
    for kw in (dict(dims=5), dict(dims=66), dict(dims=-2), dict(layout="other"), dict(axes=(16, 15)), dict(axes=()),
               dict(axes=(40, -8)), dict(base=0.0), dict(magnitude=-1.0), dict(scaling=("other", 2.0)),
               dict(scaling=("linear",)), dict(scaling=("linear", 0.0)), dict(scaling=("bands", 8.0, 2.0, 1.0, 100))):
        with pytest.raises(ValueError):
            mcs.Rotary(64, device="cpu", **kw)


def test_shapes_of_positions():
    dev = torch.device("cpu")
    p = lambda *s: torch.zeros(s, dtype=torch.int32)
    assert _position_strides(p(5), 2, 5, 1, dev) == (0, 1)
    assert _position_strides(p(2, 5), 2, 5, 1, dev) == (5, 1)
    assert _position_strides(p(2, 5, 1), 2, 5, 1, dev)[0] == 5
    assert _position_strides(p(2, 1), 2, 1, 1, dev)[0] == 1
    assert _position_strides(p(1, 5, 3), 2, 5, 3, dev)[0] == 0
    assert _position_strides(p(5, 3), 2, 5, 3, dev) == (0, 3)
    assert _position_strides(p(10, 2)[:, 0], 2, 10, 1, dev) == (0, 2)
    for bad, n, axes in ((p(4), 5, 1), (p(3, 5), 5, 1), (p(5), 5, 3), (p(2, 5, 2), 5, 3), (p(2, 5, 6)[..., ::2], 5, 3),
                         (p(5).long(), 5, 1)):
        with pytest.raises(ValueError):
            _position_strides(bad, 2, n, axes, dev)
    with pytest.raises(TypeError):
        _position_strides([0, 1], 2, 2, 1, dev)


def buffers(n=4, H=2, page=16, d=64, B=2, per=2, device="cpu"):
    e = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    return [e(n, H, page, d), e(n, H, page, d), torch.ones((n, H), device=device), torch.ones((n, H), device=device),
            torch.zeros((B, per), dtype=torch.int32, device=device)]


def test_buffers_of_a_cache():
    good = buffers()
    c = mcs.KVCache(*good)
    assert (c.capacity, c.n_pages, c.B) == (32, 4, 2)
    for i, bad in ((0, good[0][0]), (1, good[1][:3]), (1, good[1].view(torch.uint8)), (2, good[2].double()),
                   (3, good[3][:, :1]), (4, good[4].long()), (4, good[4][0]), (0, torch.zeros(4, 2, 16, 96)),
                   (4, torch.zeros((2, 4), dtype=torch.int32)[:, ::2])):
        b = list(good)
        b[i] = bad
        with pytest.raises((ValueError, TypeError)):
            mcs.KVCache(*b)
    with pytest.raises(AttributeError):
        c.page_table = good[4].clone()                               # the calls would not see it
    for bad in ((0, 2, 64), (2, 0, 64), (2, 2, 0)):
        with pytest.raises(ValueError):
            mcs.KVCache.empty(*bad, 64, device="cpu")
    with pytest.raises(ValueError):
        mcs.cache_read(c, torch.zeros(2, dtype=torch.int32), 3)      # not on a CUDA device
    with pytest.raises(TypeError):
        mcs.cache_read("cache", torch.zeros(2, dtype=torch.int32), 3)


@pytest.mark.gpu
def test_calls():
    c = mcs.KVCache(*buffers(device="cuda"))
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    rot = mcs.Rotary(64)
    three = mcs.Rotary(64, axes=(12, 10, 10))
    wide = torch.zeros((2, 2, 3, 65), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: mcs.cache_append(c, x.float(), x, i), lambda: mcs.cache_append(c, x, x[:, :, :2], i),
                lambda: mcs.cache_append(c, x[:1], x[:1], i), lambda: mcs.cache_append(c, wide[..., 1:], x, i),
                lambda: mcs.cache_append(c, x, x, i.long()), lambda: mcs.cache_append(c, x, x, None),
                lambda: mcs.cache_append(c, x, x, i, counts=i[:1]), lambda: mcs.cache_append(c, x, x, i.cpu()),
                lambda: mcs.cache_append(c, x, x, i, rotary=mcs.Rotary(128)),
                lambda: mcs.cache_append(c, x, x, i, rotary=three), lambda: mcs.cache_append(c, x, x, i, positions=i),
                lambda: mcs.cache_append(c, x, x, i, rotary=mcs.Rotary(64, dims=20)),
                lambda: mcs.cache_append(c, x, x, i, rotary=mcs.Rotary(64, device="cpu")),
                lambda: mcs.cache_read(c, i, -1), lambda: mcs.cache_read(c, None, 1), lambda: mcs.cache_read(c, i[:1], 1),
                lambda: mcs.cache_attention(x[:, :, :, :32], c, i), lambda: mcs.cache_attention(x[:1], c, i),
                lambda: mcs.cache_attention(x[:, :1], c, i), lambda: mcs.cache_attention(x.transpose(1, 2), c, i),
                lambda: mcs.cache_attention(x, c, None), lambda: mcs.cache_attention(x.half(), c, i),
                lambda: mcs.cache_attention(x, c, i, out=x[:, :1]), lambda: mcs.cache_attention(x, c, i, scale=-1.0),
                lambda: mcs.rotate(x.cpu(), i, rot), lambda: mcs.rotate(x.double(), i, rot),
                lambda: mcs.rotate(x, i, rot), lambda: mcs.rotate(x[..., ::2], i, rot),
                lambda: mcs.rotate(x, torch.zeros(3, dtype=torch.int32, device="cuda"), "rot")):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            bad()
    assert mcs.last_device_status() == 0
