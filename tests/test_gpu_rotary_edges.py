"""Rotary positions where they can go wrong beside the ordinary: numbers that are
not finite in the part of a head that stays, forward-mode derivatives, and far
positions against an exact phase."""
import math
from decimal import Decimal
from fractions import Fraction

import pytest
import torch
import torch.autograd.forward_ad as fwd

import sparse_attention_diffusion_mcs_b200 as mcs
from tests.cache_util import F64, turned
from tests.test_gpu_rotary import check

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


@pytest.mark.parametrize("layout,dims", [("half", 64), ("interleaved", 48)])
def test_forward_mode(layout, dims):
    """The map is linear in x: the tangent is turned as x is, with and without a
    gradient to x, through the gradient too (forward over backward), and a call
    that could not carry a tangent is refused."""
    rot = mcs.Rotary(64, dims=dims, layout=layout, magnitude=1.25)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, t, w, u = (torch.randn((2, 3, 9, 64), generator=g, device="cuda") for _ in range(4))
    pos = torch.randint(0, 9000, (2, 9), generator=g, device="cuda", dtype=torch.int32)
    p = pos[..., None]
    for leaf in (x, x.clone().requires_grad_(True)):
        with fwd.dual_level():
            y, dy = fwd.unpack_dual(mcs.rotate(fwd.make_dual(leaf, t), pos, rot))
            assert dy is not None
            check(y.detach(), turned(x, p, rot), torch.float32)
            check(dy.detach(), turned(t, p, rot), torch.float32)
    with fwd.dual_level(), torch.no_grad():
        dy = fwd.unpack_dual(mcs.rotate(fwd.make_dual(x, t), pos, rot)).tangent
        check(dy, turned(t, p, rot), torch.float32)
    strided = torch.randn((2, 9, 64, 3), generator=g, device="cuda").permute(0, 3, 1, 2)   # a tangent of any layout
    with fwd.dual_level():
        dy = fwd.unpack_dual(mcs.rotate(fwd.make_dual(x, strided), pos, rot)).tangent
        check(dy, turned(strided, p, rot), torch.float32)
    # the gradient's derivative along a tangent of what comes back
    leaf = x.clone().requires_grad_(True)
    with fwd.dual_level():
        y = mcs.rotate(leaf, pos, rot)
        dx, = torch.autograd.grad(y, leaf, fwd.make_dual(w, u))
        dx, ddx = fwd.unpack_dual(dx)
        check(dx, turned(w, p, rot, back=True), torch.float32)
        assert ddx is not None
        check(ddx, turned(u, p, rot, back=True), torch.float32)
    with fwd.dual_level(), pytest.raises(ValueError):
        mcs.rotate(fwd.make_dual(x, t), pos, rot, out=torch.empty_like(x))
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda z: mcs.rotate(z, pos, rot), (x,), (t,))


# 2 pi to 60 digits (the decimal expansion of pi)
TWO_PI = 2 * Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494"))


def exactly_turned(x, pos, rotary):
    """The rotation with every angle reduced in whole numbers: the turns that f
    (the rotary's own frequency) makes, less the whole ones, to 64 bits."""
    x = x.detach().to(F64).cpu().clone()
    p = rotary.dims // 2
    for i in range(p):
        j, k = (i, p + i) if rotary.layout == "half" else (2 * i, 2 * i + 1)
        turn = Fraction(rotary.frequencies[i]) / TWO_PI
        angle = torch.tensor([2 * math.pi * float(int(n) * turn % 1) for n in pos.tolist()], dtype=F64)
        c, s = torch.cos(angle), torch.sin(angle)
        a, b = x[..., j].clone(), x[..., k].clone()
        x[..., j], x[..., k] = a * c - b * s, a * s + b * c
    return x


@pytest.mark.parametrize("layout,dims", [("half", 128), ("interleaved", 128), ("half", 22)])
def test_far_positions_against_an_exact_phase(layout, dims):
    """Every 32-bit position.  Of a pair (a, b), fp32 throughout: the phase is cut to
    2^-32 turns (1.5e-9 rad) and the table's fraction is off by pos * 2^-65 turns
    (less still); sine and cosine are off by 1.1e-7 each (the polynomials), 1.6e-7
    of the pair's length together; one product and the sum are rounded, 2^-24 of
    that length each, 1.2e-7, the second being the output's own.  2.9e-7 in all."""
    rot = mcs.Rotary(128, dims=dims, layout=layout, base=500000.0)
    g = torch.Generator(device="cuda").manual_seed(7)
    far = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, -2 ** 30 - 77, 2 ** 24 + 1, 123456789, 0, 1, -1, 131071]
    pos = torch.tensor(far, dtype=torch.int32, device="cuda")
    x = torch.randn((1, 3, len(far), 128), generator=g, device="cuda")
    ref = exactly_turned(x, pos, rot)
    got = mcs.rotate(x, pos, rot).cpu().to(F64)
    p = dims // 2
    a, b = (x[..., :p], x[..., p:dims]) if layout == "half" else (x[..., 0:dims:2], x[..., 1:dims:2])
    length = torch.hypot(a, b).cpu().to(F64)
    err = (got - ref).abs()
    e0, e1 = (err[..., :p], err[..., p:dims]) if layout == "half" else (err[..., 0:dims:2], err[..., 1:dims:2])
    tol = 2.9e-7 * length
    assert (e0 <= tol).all() and (e1 <= tol).all()
    assert torch.equal(got[..., dims:], x[..., dims:].cpu().to(F64))
