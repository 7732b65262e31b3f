"""Outputs that lie over inputs are refused before any launch: threads would read
what others have written.  (No GPU needed: the library's own checks, and the
Python calls' beside them.)"""
import ctypes

import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs
from sparse_attention_diffusion_mcs_b200 import _lib
from sparse_attention_diffusion_mcs_b200 import build as _build
from sparse_attention_diffusion_mcs_b200.rotary import _check_apart
from tests.test_cache_refusals import FAKE, INVALID, I64x3, cache, rotary

X = 0x1000000


@pytest.fixture(scope="module")
def L():
    _build.build()
    return _lib.lib()


@pytest.mark.parametrize("dtype,size", [(0, 2), (2, 4)])
def test_rotate(L, dtype, size):
    B, H, N, d = 2, 3, 5, 64

    def call(out, strides=(H * N * d, N * d, d)):
        return L.mcs_rotate(X, dtype, B, H, N, d, I64x3(*strides), FAKE, 0, 1, rotary(), 0, out, None)
    n = B * H * N * d * size
    for out in (X + size, X - size, X + n - size, X - n + size, X + 16, X - 16):
        assert call(out) == INVALID
    wide = (N * H * d, d, H * d)                                 # a projection's layout over the same memory
    assert call(X, wide) == INVALID
    spread = (4 * H * N * d, N * d, d)                           # reaches further than the output does
    for out in (X, X + 4 * n // 2, X + (4 * H * N * d + H * N * d) * size - size, X - n + size):
        assert call(out, spread) == INVALID


def test_attention(L):
    B, Hq, Nq, d = 2, 4, 3, 64
    n = B * Hq * Nq * d * 2
    for out in (X, X + 16, X - 16, X + n - 16, X - n + 16):
        assert L.mcs_cache_attention(cache(), X, Hq, Nq, FAKE, None, 0, 0.125, out, None, FAKE, 2 ** 30, None) == INVALID


def test_python_calls_say_why():
    base = torch.zeros(4000, dtype=torch.bfloat16)
    x = base[:1920].view(2, 3, 5, 64)
    for out in (base[8:1928].view(2, 3, 5, 64), base[1919:3839].view(2, 3, 5, 64)):
        with pytest.raises(ValueError, match="overlap"):
            _check_apart(x, out, False)
    _check_apart(x, base[1920:3840].view(2, 3, 5, 64), False)
    with pytest.raises(ValueError, match="overlap"):
        _check_apart(x, x, False)
    _check_apart(x, x, True)                                     # in place
    with pytest.raises(ValueError, match="overlap"):
        _check_apart(base[:1920].view(2, 5, 3, 64).transpose(1, 2), x, True)
    _check_apart(x[:0], x[:0], False)


@pytest.mark.gpu
def test_calls_on_the_gpu():
    rot = mcs.Rotary(64, dims=48, layout="interleaved")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    qkv = torch.randn((1, 5, 6, 64), device="cuda").to(torch.bfloat16)
    x = qkv[:, :, :2].transpose(1, 2)
    with pytest.raises(ValueError, match="overlap"):
        mcs.rotate(x, pos, rot, out=qkv.view(-1)[:640].view(1, 2, 5, 64))
    for dtype, dims in ((torch.bfloat16, 48), (torch.float32, 50), (torch.float16, 22)):
        rot = mcs.Rotary(64, dims=dims, layout="interleaved")
        z = torch.randn((2, 19, 5, 64), device="cuda").to(dtype)
        want = mcs.rotate(z, pos, rot)
        assert mcs.rotate(z, pos, rot, out=z) is z and torch.equal(z, want)      # in place
    c = mcs.KVCache.empty(1, 2, 64, 64)
    n = torch.tensor([3], dtype=torch.int32, device="cuda")
    Q = torch.randn((2, 2, 5, 64), device="cuda").to(torch.bfloat16)
    with pytest.raises(ValueError, match="overlap"):
        mcs.cache_attention(Q[:1], c, n, out=Q[:1])
    mcs.cache_attention(Q[:1], c, n, out=Q[1:])
