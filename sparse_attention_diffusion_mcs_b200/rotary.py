"""Rotary positions: the step that turns a projection's queries and keys by
their positions before any attention entry sees them, from any strided
[B, H, N, d] view to the contiguous layout those entries take.

``Rotary`` describes which numbers of a head turn and how fast; ``rotate``
applies it (CUDA library, include/mcs.h: mcs_rotate) and is differentiable in
x: the gradient is the same kernel turning back.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd import forward_ad

from . import api
from ._lib import McsRotary, check, lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I64x3 = ctypes.c_int64 * 3
# the current stream's handle without the objects around it (a call takes a few microseconds, they cost two)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(name: str, device, *args) -> None:
    """The library function on `device`'s current stream, with that device current."""
    index = device.index
    if index == torch.cuda.current_device():
        code = getattr(lib(), name)(*args, _raw_stream(index))
    else:
        with api._on(device):
            code = getattr(lib(), name)(*args, _raw_stream(index))
    if code:
        check(code, name)


class _Handle:
    """What the library holds the addresses of: another tensor under the name would
    not be seen, and the old one's memory would be read after it is freed."""

    _held = frozenset()

    def _hold(self):
        self._held = frozenset((*self.__dict__, "_held"))

    def __setattr__(self, name, value):
        if name in self._held:
            raise AttributeError(f"{name} is fixed: make another {type(self).__name__}")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        if name in self._held:
            raise AttributeError(f"{name} is fixed: make another {type(self).__name__}")
        super().__delattr__(name)


class Rotary(_Handle):
    """Which numbers of a head of size d turn with the position, and how fast.

    dims: how many (from the first; even), default all d.
    layout: "half" pairs (i, dims/2 + i), "interleaved" pairs (2i, 2i + 1).
    axes: pairs per position axis, summing to dims/2 (e.g. time, row, column);
      default one axis.  Within an axis of m pairs, pair j turns by
      base^(-j/m) radians per position.
    scaling, for contexts longer than a model was trained on:
      ("linear", factor): every frequency divided by factor;
      ("ntk", factor): base raised to base * factor^(m/(m-1)), so that the
        slowest pair slows down by factor and the fastest stays;
      ("bands", factor, low, high, original): by the turns a pair makes over
        `original` positions: from `high` turns on it stays, up to `low` it is
        divided by factor, linear in between.
    magnitude: factor on the rotated numbers.
    A rotary is fixed: for other numbers make another one.
    """

    def __init__(self, d: int, dims: Optional[int] = None, base: float = 10000.0, layout: str = "half",
                 axes: Optional[Sequence[int]] = None, scaling: Optional[Tuple] = None, magnitude: float = 1.0,
                 device="cuda"):
        dims = d if dims is None else int(dims)
        if d < 1 or dims < 0 or dims % 2 or dims > d:
            raise ValueError(f"dims must be even and in [0, d]: got {dims} of {d}")
        if layout not in ("half", "interleaved"):
            raise ValueError(f'layout is "half" or "interleaved", got {layout!r}')
        axes = [dims // 2] if axes is None else [int(m) for m in axes]
        if not axes or any(m < 0 for m in axes) or sum(axes) != dims // 2:
            raise ValueError(f"axes must sum to dims/2 = {dims // 2}: got {axes}")
        if not (base > 0 and math.isfinite(base)) or not (magnitude > 0 and math.isfinite(magnitude)):
            raise ValueError("base and magnitude must be positive and finite")
        self.d, self.dims, self.base, self.layout, self.axes = int(d), dims, float(base), layout, tuple(axes)
        self.scaling, self.magnitude = scaling, float(magnitude)
        self.frequencies = [f for m in axes for f in _frequencies(m, float(base), scaling)]
        # fractions of a turn per position, times 2^64, kept in int64's bits
        turns = [_turns(f) % 2 ** 64 for f in self.frequencies]
        turns = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
        axis = [a for a, m in enumerate(axes) for _ in range(m)]
        # one copy to the device: the turns' 64-bit numbers, then the axes' 32-bit ones
        both = torch.cat([torch.tensor(turns, dtype=torch.int64).view(torch.int32), torch.tensor(axis, dtype=torch.int32)])
        both = both.to(device)
        self.turns, self.axis = both[:dims].view(torch.int64), both[dims:]
        self.device = both.device
        self._c = McsRotary(self.turns.data_ptr(), self.axis.data_ptr(), dims // 2, int(layout == "interleaved"),
                            len(axes), float(magnitude))
        self._ref = ctypes.byref(self._c)
        self._hold()


# pi * 10^59; in 53 bits the fractions below would be off by hundreds, which far positions multiply
_PI = 314159265358979323846264338327950288419716939937510582097494


def _turns(f: float) -> int:
    """round(f / 2 pi * 2^64), in whole numbers."""
    num, den = f.as_integer_ratio()
    num, den = num * 2 ** 64 * 10 ** 59, den * 2 * _PI
    return (2 * num + den) // (2 * den)


def _frequencies(m: int, base: float, scaling: Optional[Tuple]):
    """Radians per position of the m pairs of one axis."""
    kind = scaling[0] if scaling else None
    if kind not in (None, "linear", "ntk", "bands"):
        raise ValueError(f"unknown scaling {kind!r}")
    if kind and len(scaling) != (5 if kind == "bands" else 2):
        raise ValueError(f"scaling {kind!r} takes {4 if kind == 'bands' else 1} number(s)")
    if kind and not all(x > 0 and math.isfinite(x) for x in scaling[1:]):
        raise ValueError("scaling numbers must be positive and finite")
    if kind == "bands" and not scaling[3] > scaling[2]:
        raise ValueError("scaling bands: high must exceed low")
    if kind == "ntk" and m > 1:
        base = base * scaling[1] ** (m / (m - 1))
    f = [base ** (-j / m) for j in range(m)]
    if kind == "linear":
        f = [x / scaling[1] for x in f]
    if kind == "bands":
        _, factor, low, high, original = scaling
        keep = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        f = [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]
    return f


def _position_strides(positions: torch.Tensor, B: int, N: int, axes: int, device) -> Tuple[int, int]:
    """(stride over B, stride over N) of int32 positions [N] or [B, N] (one
    axis), [N, axes] or [B, N, axes]; a B of 1 is repeated."""
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a tensor")
    if positions.dtype != torch.int32 or positions.device != device:
        raise ValueError(f"positions must be an int32 tensor on {device}, got {positions.dtype} on {positions.device}")
    shape, stride = tuple(positions.shape), positions.stride()
    if shape == (B, N, axes) and (axes == 1 or stride[2] == 1):
        return (0 if B == 1 else stride[0]), stride[1]
    if axes == 1 and shape and shape[-1] != 1 or axes == 1 and len(shape) == 1:
        shape, stride = shape + (1,), stride + (1,)
    elif axes == 1 and len(shape) == 2 and N == 1 and shape[0] == B:      # [B, 1]: one token of each sequence
        shape, stride = shape + (1,), stride + (1,)
    if len(shape) == 2:
        shape, stride = (1,) + shape, (0,) + stride
    if len(shape) != 3 or shape[0] not in (1, B) or shape[1:] != (N, axes):
        raise ValueError(f"positions must be [{N}, {axes}] or [{B}, {N}, {axes}] (the last may be left out for one "
                         f"axis), got {tuple(positions.shape)}")
    if axes > 1 and stride[2] != 1:
        raise ValueError("the axes of positions must be contiguous")
    return (0 if shape[0] == 1 else stride[0]), stride[1]


def _check_rotary(rotary: "Rotary", d: int, device):
    if not isinstance(rotary, Rotary):
        raise TypeError("rotary must be a Rotary")
    if rotary.d != d:
        raise ValueError(f"rotary is for heads of {rotary.d}, the tensor's have {d}")
    if rotary.device != device:
        raise ValueError(f"rotary is on {rotary.device}, the tensor on {device}")


def _launch(x: torch.Tensor, positions: torch.Tensor, pos_b: int, pos_n: int, rotary: Rotary, back: int,
            out: torch.Tensor) -> None:
    B, H, N, d = x.shape
    sb, sh, sn, _ = x.stride()
    _run("mcs_rotate", x.device, x.data_ptr(), _DTYPES[x.dtype], B, H, N, d, _I64x3(sb, sh, sn), positions.data_ptr(),
         pos_b, pos_n, rotary._ref, back, out.data_ptr())


def _check_apart(x: torch.Tensor, out: torch.Tensor, in_place: bool) -> None:
    """out (contiguous, x's shape) shares no memory with the stretch from x's first
    to its last number, or (in_place) is x itself: threads would read what others
    have written."""
    n, apart = x.numel(), out.data_ptr() - x.data_ptr()
    packed = x.is_contiguous()
    if n == 0 or in_place and packed and apart == 0:
        return
    end = n if packed else sum((m - 1) * s for m, s in zip(x.shape, x.stride())) + 1
    if -n < apart / x.element_size() < end:
        raise ValueError("out must not overlap the input")


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x with its last dimension contiguous (a gradient may come in any layout)."""
    return x if x.stride(3) == 1 or x.shape[3] == 1 else x.contiguous()


def _empty(x: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _differentiated(x: torch.Tensor) -> bool:
    """Whether a gradient or a tangent (forward mode) goes through x."""
    if torch.is_grad_enabled() and x.requires_grad:
        return True
    # (no level is open: no tangents; unpack_dual alone would take 0.4 us to say so)
    return getattr(forward_ad, "_current_level", 0) >= 0 and forward_ad.unpack_dual(x).tangent is not None


def _turned(x: torch.Tensor, positions: torch.Tensor, pos_b: int, pos_n: int, rotary: Rotary, back: int) -> torch.Tensor:
    """x (its last dimension contiguous) turned, differentiably where x is."""
    if _differentiated(x):
        return _Rotate.apply(x, positions, pos_b, pos_n, rotary, back)
    out = _empty(x)
    _launch(x, positions, pos_b, pos_n, rotary, back, out)
    return out


class _Rotate(torch.autograd.Function):
    """Turning by the positions, or back; the gradient is the other one, and the
    tangent of x is turned as x is."""

    @staticmethod
    def forward(ctx, x, positions, pos_b, pos_n, rotary, back):
        out = _empty(x)
        _launch(x, positions, pos_b, pos_n, rotary, back, out)
        ctx.save_for_backward(positions)
        ctx.save_for_forward(positions)
        ctx.more = (pos_b, pos_n, rotary)
        ctx.back = back
        return out

    @staticmethod
    def backward(ctx, grad):
        positions, = ctx.saved_tensors
        return _turned(_rows(grad), positions, *ctx.more, 1 - ctx.back), None, None, None, None, None

    @staticmethod
    def jvp(ctx, tangent, *_):
        positions, = ctx.saved_tensors
        return _turned(_rows(tangent), positions, *ctx.more, ctx.back)


def rotate(x: torch.Tensor, positions: torch.Tensor, rotary: Rotary, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [B, H, N, d] (bf16, fp16 or fp32, any strides over B, H and N) with its
    pairs turned by the tokens' positions: contiguous [B, H, N, d].

    positions: int32 [N] or [B, N], with several axes [N, axes] or
    [B, N, axes].  Differentiable in x (not with `out`), any number of times,
    backward and in forward mode.  `out` may be x itself, contiguous (in place),
    and must not overlap it otherwise.

    To capture a backward pass into a CUDA graph while an eager graph of the same
    leaf lives, run the eager one on the capturing stream: torch ties a leaf's
    gradient to the stream of its first use, and the capture fails otherwise."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.dtype not in _DTYPES or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor [B, H, N, d] of bf16, fp16 or fp32")
    B, H, N, d = x.shape
    _check_rotary(rotary, d, x.device)
    pos_b, pos_n = _position_strides(positions, B, N, len(rotary.axes), x.device)
    if x.stride(3) != 1 and d > 1:
        raise ValueError("the last dimension of x must be contiguous")
    if out is None:
        return _turned(x, positions, pos_b, pos_n, rotary, 0)
    if _differentiated(x):
        raise ValueError("rotate with a gradient writes its own output: leave `out` away")
    api._check_tensor(out, "out", x.shape, x.dtype, x.device)
    _check_apart(x, out, True)
    _launch(x, positions, pos_b, pos_n, rotary, 0, out)
    return out
