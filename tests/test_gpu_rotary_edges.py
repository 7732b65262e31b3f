"""Rotary positions where they can go wrong beside the ordinary: numbers that are
not finite in the part of a head that stays."""
import math

import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int32 if x.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d,dims,layout", [(128, 64, "half"), (64, 16, "half"), (64, 50, "interleaved"),
                                           (64, 16, "interleaved"), (128, 0, "interleaved"), (64, 22, "half")])
def test_numbers_that_stay_keep_their_bits(dtype, d, dims, layout):
    """Behind the turned part inf, NaN and -0 come out as they went in and reach
    no neighbour, whatever the alignment (which chooses the kernel), forward and
    back; the turned part is what it is without them."""
    B, H, N = 2, 3, 37
    rot = mcs.Rotary(d, dims=dims, layout=layout)
    g = torch.Generator(device="cuda").manual_seed(d + dims)
    pos = torch.randint(0, 5000, (N,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((B, H, N, d), generator=g, device="cuda").to(dtype)
    plain = x.clone()
    for j, v in ((dims, math.inf), (dims + 3, -math.inf), (d - 2, math.nan), (d - 7, -0.0), (d - 6, -1.0), (d - 13, -0.0)):
        x[:, :, j % 5::5, j] = v
    wide = torch.empty(B * H * N * d + 1, dtype=dtype, device="cuda")
    odd = wide[1:].view(B, H, N, d)                       # rows off 16 bytes
    odd.copy_(x)
    for y, ref in ((mcs.rotate(x, pos, rot), mcs.rotate(plain, pos, rot)), (mcs.rotate(odd, pos, rot), None)):
        assert torch.equal(bits(y[..., dims:].contiguous()), bits(x[..., dims:].contiguous()))
        if ref is not None:
            assert torch.equal(bits(y[..., :dims].contiguous()), bits(ref[..., :dims].contiguous()))
            first = y
        else:
            assert torch.equal(bits(y), bits(first))
    leaf = torch.zeros_like(x, requires_grad=True)
    dx, = torch.autograd.grad(mcs.rotate(leaf, pos, rot), leaf, x)
    assert torch.equal(bits(dx[..., dims:].contiguous()), bits(x[..., dims:].contiguous()))
    assert torch.isfinite(dx[..., :dims]).all()
