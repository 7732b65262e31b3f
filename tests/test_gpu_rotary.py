"""Rotary positions against the definition in 64 bits: layouts, axes, parts of
the head, types, far and negative positions, strides, and the gradient.

Bound per number: the phase's rounding to fp32 (2^-25 half turns, 9.4e-8 rad),
sincospif's (2 ulp, 1.2e-7) and two fp32 roundings of the sum (2 * 2^-24), on
the pair's length: 3.4e-7; the pair's length is at most sqrt(2) * the largest
number: 5e-7.  Then half a step of the type."""
import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs
from tests.cache_util import F64, turned

pytestmark = pytest.mark.gpu


def check(got, ref, dtype):
    half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0       # half of fp16's smallest step
    tol = half * ref.abs() + 5e-7 * ref.abs().max() * (1 + half) + tiny
    assert got.dtype == dtype and got.is_contiguous()
    assert ((got.cpu().to(F64) - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d,dims,layout,axes,scaling,first", [
    (128, 128, "half", None, None, 0), (128, 96, "half", None, ("linear", 4.0), 7), (64, 64, "interleaved", None, None, 0),
    (64, 48, "interleaved", (8, 9, 7), ("ntk", 2.0), 100), (128, 128, "half", (22, 21, 21), None, 0),
    (64, 32, "half", None, ("bands", 8.0, 1.0, 32.0, 512), 2 ** 31 - 200), (128, 0, "half", None, None, 3),
    (64, 22, "half", None, None, -1000), (80, 80, "half", None, None, 5), (50, 50, "interleaved", None, None, 5),
    (6, 2, "half", None, None, 9), (2, 2, "interleaved", None, None, 9), (48, 16, "half", (8, 0), None, 3)])
def test_matches_the_definition(dtype, d, dims, layout, axes, scaling, first):
    B, H, N = 2, 5, 67
    g = torch.Generator(device="cuda").manual_seed(d + dims)
    rot = mcs.Rotary(d, dims=dims, layout=layout, axes=axes, scaling=scaling, magnitude=1.25)
    x = torch.randn((B, N, H, d), generator=g, device="cuda").to(dtype).transpose(1, 2)
    n = len(rot.axes)
    pos = torch.randint(0, 200, (B, N, n), generator=g, device="cuda", dtype=torch.int32) + first
    check(mcs.rotate(x, pos, rot), turned(x, pos, rot), dtype)
    # one row of positions for every sequence; for one axis, without the axis
    one = pos[:1].expand(B, -1, -1)
    flat = pos[0, :, 0].contiguous() if n == 1 else pos[0].contiguous()
    assert torch.equal(mcs.rotate(x, flat, rot), mcs.rotate(x, one.contiguous(), rot))


@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (3, 24, 1), (1, 2, 4099), (0, 3, 4), (2, 0, 4), (2, 3, 0)])
def test_sizes_from_none_to_many(B, H, N):
    rot = mcs.Rotary(64)
    x = torch.randn((B, H, N, 64), device="cuda").to(torch.bfloat16)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None].expand(B, N) if B else torch.zeros((1, N), dtype=torch.int32, device="cuda")
    y = mcs.rotate(x, pos, rot)
    assert y.shape == x.shape
    if x.numel():
        check(y, turned(x, pos[..., None], rot), torch.bfloat16)


def test_strides_and_alignment():
    """Every view with a contiguous last dimension, aligned or not, broadcast ones too, gives the same bits."""
    rot = mcs.Rotary(64, layout="half")
    base = torch.randn(200_000, device="cuda").to(torch.bfloat16)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    for x in (torch.as_strided(base, (2, 3, 9, 64), (3000, 70, 300, 1), 0), torch.as_strided(base, (2, 3, 9, 64), (3000, 72, 304, 1), 3),
              torch.as_strided(base, (2, 3, 9, 64), (4096, 64, 192, 1), 8), base[:64].expand(2, 3, 9, 64),
              torch.as_strided(base, (1, 3, 9, 64), (5, 64, 192, 1), 0)):
        y = mcs.rotate(x, pos, rot)
        check(y, turned(x, pos[None, :, None].expand(x.shape[0], -1, -1), rot), torch.bfloat16)
        out = torch.empty(x.shape, dtype=x.dtype, device="cuda")
        assert mcs.rotate(x, pos, rot, out=out) is out and torch.equal(out, y)


@pytest.mark.parametrize("layout,dims,axes", [("half", 64, (12, 10, 10)), ("interleaved", 48, None), ("half", 22, None)])
def test_gradient(layout, dims, axes):
    """Against the formula (turning back), and against differences: the map is
    linear, so <grad, R(e)> is the derivative along e exactly."""
    rot = mcs.Rotary(64, dims=dims, layout=layout, axes=axes, magnitude=0.75)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((2, 7, 3, 64), generator=g, device="cuda").transpose(1, 2).requires_grad_(True)
    pos = torch.randint(0, 50000, (2, 7, len(rot.axes)), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn((2, 3, 7, 64), generator=g, device="cuda")
    y = mcs.rotate(x, pos, rot)
    dx, = torch.autograd.grad(y, x, w)
    check(dx, turned(w, pos, rot, back=True), torch.float32)
    e = torch.randn(x.shape, generator=g, device="cuda")
    with torch.no_grad():
        step = mcs.rotate((x + e), pos, rot).double() - mcs.rotate((x - e), pos, rot).double()
    along = 0.5 * (step * w.double()).sum().item()
    assert abs(along - (dx.double() * e.double()).sum().item()) <= 2e-6 * (w.double().norm() * e.double().norm()).item()


def test_gradient_of_a_gradient():
    """The gradient is linear in what comes back, so its gradient turns forward again."""
    rot = mcs.Rotary(64, dims=48)
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 1001
    x, w, e = (torch.randn((1, 2, 9, 64), device="cuda", requires_grad=True) for _ in range(3))
    dx, = torch.autograd.grad(mcs.rotate(x, pos, rot), x, w, create_graph=True)
    dw, = torch.autograd.grad(dx, w, e)
    check(dw, turned(e, pos[None, :, None], rot), torch.float32)


def test_gradient_of_a_broadcast_input_and_of_any_layout():
    rot = mcs.Rotary(64)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    leaf = torch.randn((1, 1, 5, 64), device="cuda", requires_grad=True)
    y = mcs.rotate(leaf.expand(2, 3, 5, 64), pos, rot)
    w = torch.randn((2, 3, 64, 5), device="cuda").transpose(2, 3)       # last dimension not contiguous
    y.backward(w)
    ref = turned(w, pos[None, :, None].expand(2, -1, -1), rot, back=True).sum((0, 1), keepdim=True)
    assert ((leaf.grad.cpu().to(F64) - ref).abs() <= 6 * 5e-7 * w.abs().max().item() + 5 * 2.0 ** -24 * ref.abs()).all()
    y = mcs.rotate(leaf.expand(2, 3, 5, 64), pos, rot)
    y.sum().backward()                                                    # a gradient of stride 0
    with pytest.raises(ValueError):
        mcs.rotate(leaf, pos, rot, out=torch.empty_like(leaf))


def test_captured_forward_and_backward_beside_an_eager_one():
    """A step captured while an eager graph of the same leaf lives, replayed on
    new values.  The eager one ran on the capturing stream: torch ties a leaf's
    gradient to the stream of its first use, for every differentiable operator."""
    rot = mcs.Rotary(128)
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    x = torch.randn((1, 2, 33, 128), device="cuda", requires_grad=True)
    w = torch.randn((1, 2, 33, 128), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alive = mcs.rotate(x, pos, rot)
        torch.autograd.grad(mcs.rotate(x, pos, rot), x, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = mcs.rotate(x, pos, rot)
        dx, = torch.autograd.grad(y, x, w)
    with torch.no_grad():
        x.copy_(torch.randn_like(x))
        w.copy_(torch.randn_like(w))
        pos += 1000
    graph.replay()
    p = pos[None, :, None]
    check(y.detach(), turned(x, p, rot), torch.float32)
    check(dx, turned(w, p, rot, back=True), torch.float32)
    assert alive.shape == x.shape


def test_another_stream():
    rot = mcs.Rotary(64)
    pos = torch.arange(3000, dtype=torch.int32, device="cuda")
    x = torch.randn((1, 8, 3000, 64), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = mcs.rotate(x, pos, rot)
    s.synchronize()
    check(y, turned(x, pos[None, :, None], rot), torch.float32)
