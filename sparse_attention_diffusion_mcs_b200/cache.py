"""A paged cache of keys and values held in 8 bits, and attention over it.

A model that generates chunk by chunk keeps the keys and values of what is
finished and attends to them from each new chunk.  ``KVCache`` holds them in
pages of e4m3 numbers with one power-of-two scale per (page, head);
``cache_append`` adds tokens (keys rotated on the way), ``cache_read`` gives
tokens back as the bf16 tensors that ``plan`` and ``dense`` take, and
``cache_attention`` attends to them.  Lengths and places stay on the device
and belong to the caller, so every call can be captured into a CUDA graph.
Kernels and conventions: include/mcs.h.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import api
from ._lib import McsCache, lib
from .rotary import Rotary, _check_apart, _check_rotary, _Handle, _position_strides, _run

_I64x3 = ctypes.c_int64 * 3


class KVCache(_Handle):
    """The cache's buffers: k_pages, v_pages float8_e4m3fn [n_pages, H, page, d],
    k_scale, v_scale float32 [n_pages, H], page_table int32 [B, max_pages].
    Token j of sequence b is slot j % page of page page_table[b, j // page].
    A number stands for e4m3 * scale of its page and head.  Scales of a caller's own
    are 0 to 2^90 for keys, 2^-90 to 2^90, or 0, for values; attention leaves out,
    and records (last_device_status), a page whose scale is none of these.

    Calls work on these very buffers: change their contents in place (new pages
    in page_table, for instance); for other buffers make another KVCache."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 page_table: torch.Tensor):
        if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
            raise ValueError("k_pages must be a tensor [n_pages, H, page, d]")
        n_pages, H, page, d = k_pages.shape
        dev = k_pages.device
        if d not in (64, 128) or page not in (16, 32, 64, 128):
            raise ValueError(f"d must be 64 or 128 and page 16, 32, 64 or 128: got d {d}, page {page}")
        api._check_tensor(k_pages, "k_pages", (n_pages, H, page, d), torch.float8_e4m3fn, dev)
        api._check_tensor(v_pages, "v_pages", (n_pages, H, page, d), torch.float8_e4m3fn, dev)
        api._check_tensor(k_scale, "k_scale", (n_pages, H), torch.float32, dev)
        api._check_tensor(v_scale, "v_scale", (n_pages, H), torch.float32, dev)
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be a tensor [B, max_pages]")
        B, max_pages = page_table.shape
        api._check_tensor(page_table, "page_table", (B, max_pages), torch.int32, dev)
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.page_table = page_table
        self.B, self.H, self.d, self.page = B, H, d, page
        self.n_pages, self.max_pages, self.device = n_pages, max_pages, dev
        self._c = McsCache(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                           page_table.data_ptr(), n_pages, max_pages, B, H, page, d)
        self._ref = ctypes.byref(self._c)
        self._hold()

    @property
    def capacity(self) -> int:
        """Tokens that a sequence's row of the table has places for."""
        return self.max_pages * self.page

    @staticmethod
    def empty(B: int, H: int, capacity: int, d: int, page: int = 64, device="cuda") -> "KVCache":
        """A cache with room for `capacity` tokens of each of B sequences, the
        pages dealt out in order."""
        if B < 1 or H < 1 or capacity < 1:
            raise ValueError(f"B, H and capacity must be positive: got {B}, {H}, {capacity}")
        per = -(-int(capacity) // page)
        n = B * per
        pages = [torch.zeros((n, H, page, d), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                 for _ in range(2)]
        scales = [torch.full((n, H), 2.0 ** -60, dtype=torch.float32, device=device) for _ in range(2)]
        table = torch.arange(n, dtype=torch.int32, device=device).view(B, per)
        return KVCache(*pages, *scales, table)


def _per_sequence(t: Optional[torch.Tensor], name: str, cache: KVCache) -> int:
    """The address of an int32 [B] tensor (0 for None)."""
    if t is None:
        return 0
    api._check_tensor(t, name, (cache.B,), torch.int32, cache.device)
    return t.data_ptr()


def _check_cache(cache: KVCache):
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    if cache.device.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")


def _row_strides(t: torch.Tensor, name: str):
    """t's strides over B, H and n, with rows that can be read 16 bytes at a time."""
    (b, h, n, _), (sb, sh, sn, sd) = t.shape, t.stride()
    if sd != 1 or t.data_ptr() % 16 or (sb % 8 and b > 1) or (sh % 8 and h > 1) or (sn % 8 and n > 1):
        raise ValueError(f"{name}'s rows must be contiguous and start on 16-byte boundaries")
    return _I64x3(sb, sh, sn)


def cache_append(cache: KVCache, K: torch.Tensor, V: torch.Tensor, start: torch.Tensor,
                 counts: Optional[torch.Tensor] = None, rotary: Optional[Rotary] = None,
                 positions: Optional[torch.Tensor] = None) -> None:
    """Put K, V (bf16 [B, H, n, d], strided views welcome: the last dimension
    contiguous, rows on 16-byte boundaries) at places start[b] .. of each
    sequence (start int32 [B]; counts int32 [B]: how many of the n, default
    all), where the sequence then ends.

    rotary: keys are turned on the way, by `positions` (as in `rotate`) or by
    their places.  No gradient flows into the cache."""
    _check_cache(cache)
    for t, name in ((K, "K"), (V, "V")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.device != cache.device or t.dim() != 4:
            raise ValueError(f"{name} must be a bf16 tensor [B, H, n, d] on {cache.device}")
    n = K.shape[2]
    if tuple(K.shape) != (cache.B, cache.H, n, cache.d) or K.shape != V.shape:
        raise ValueError(f"K and V must be [{cache.B}, {cache.H}, n, {cache.d}], got {tuple(K.shape)} and {tuple(V.shape)}")
    if n == 0:
        return
    ks, vs = _row_strides(K, "K"), _row_strides(V, "V")
    if start is None:
        raise TypeError("start must be a tensor")
    at = _per_sequence(start, "start", cache)
    how_many = _per_sequence(counts, "counts", cache)
    rot, pos, pos_b, pos_n = None, 0, 0, 0
    if rotary is not None:
        _check_rotary(rotary, cache.d, cache.device)
        if rotary.layout == "half" and rotary.dims % 16:
            raise ValueError("appending with the half layout rotates a multiple of 16 numbers")
        if positions is not None:
            pos_b, pos_n = _position_strides(positions, cache.B, n, len(rotary.axes), cache.device)
            pos = positions.data_ptr()
        elif len(rotary.axes) != 1:
            raise ValueError("several position axes need `positions`")
        rot = rotary._ref
    elif positions is not None:
        raise ValueError("positions without rotary")
    _run("mcs_cache_append", cache.device, cache._ref, K.data_ptr(), V.data_ptr(), ks, vs, n, at, how_many, pos, pos_b, pos_n,
         rot)


def cache_read(cache: KVCache, start: torch.Tensor, n: int,
               counts: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Tokens start[b] .. start[b] + n - 1 of each sequence: K, V bf16
    [B, H, n, d]; rows from counts[b] on and behind the table are zeros."""
    _check_cache(cache)
    n = int(n)
    if n < 0:
        raise ValueError("n must not be negative")
    if start is None:
        raise TypeError("start must be a tensor")
    at = _per_sequence(start, "start", cache)
    how_many = _per_sequence(counts, "counts", cache)
    K = torch.empty((cache.B, cache.H, n, cache.d), dtype=torch.bfloat16, device=cache.device)
    V = torch.empty_like(K)
    _run("mcs_cache_read", cache.device, cache._ref, at, how_many, n, K.data_ptr(), V.data_ptr())
    return K, V


def cache_attention(Q: torch.Tensor, cache: KVCache, lengths: torch.Tensor, causal: bool = False,
                    counts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, return_lse: bool = False):
    """Attention of Q (bf16 [B, Hq, Nq, d], Hq a multiple of the cache's H) to
    the first lengths[b] (int32 [B]) tokens of each sequence: bf16 O
    [B, Hq, Nq, d], or (O, lse float32 [B, Hq, Nq]).

    causal: query i of a sequence stands at place lengths[b] - counts[b] + i
    and sees the places up to its own.  counts (int32 [B], default Nq): query
    tokens of each sequence; rows behind give zeros, as rows do that see
    nothing (lse -inf).  A query that is not finite gives NaN, and so does a row
    all of whose scores lie beyond fp32's range.  `out` must not
    overlap Q.  For inference: no gradient flows through the cache."""
    _check_cache(cache)
    if not isinstance(Q, torch.Tensor) or Q.dim() != 4:
        raise ValueError("Q must be a tensor [B, Hq, Nq, d]")
    B, Hq, Nq, d = Q.shape
    if B != cache.B or d != cache.d or Hq < 1 or Hq % cache.H:
        raise ValueError(f"Q must be [{cache.B}, a multiple of {cache.H}, Nq, {cache.d}], got {tuple(Q.shape)}")
    api._check_tensor(Q, "Q", Q.shape, torch.bfloat16, cache.device)
    if lengths is None:
        raise TypeError("lengths must be a tensor")
    kept = _per_sequence(lengths, "lengths", cache)
    how_many = _per_sequence(counts, "counts", cache)
    if out is None:
        out = torch.empty_like(Q)
    else:
        api._check_tensor(out, "out", Q.shape, torch.bfloat16, cache.device)
        _check_apart(Q, out, False)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=cache.device) if return_lse else None
    need = lib().mcs_cache_attention_workspace_size(cache._ref, Hq, Nq)
    ws = torch.empty(need, dtype=torch.uint8, device=cache.device) if need else None
    _run("mcs_cache_attention", cache.device, cache._ref, Q.data_ptr(), Hq, Nq, kept, how_many, int(causal),
         api._scale(d, scale), out.data_ptr(), 0 if lse is None else lse.data_ptr(), 0 if ws is None else ws.data_ptr(), need)
    return (out, lse) if return_lse else out
