"""The cache where it can go wrong beside the ordinary: numbers that are not
finite in the part of a key that stays."""
import math

import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs
from tests.cache_util import F64, tokens
from tests.test_gpu_cache import i32

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
