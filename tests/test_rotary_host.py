"""Rotary's tables on the host: the library holds their addresses, so they cannot
be rebound, and the turns are the nearest 64-bit fractions."""
import copy
from decimal import Decimal
from fractions import Fraction

import pytest
import torch

import sparse_attention_diffusion_mcs_b200 as mcs


def test_what_the_library_holds_cannot_be_rebound():
    """The addresses of turns and axis and a copy of the numbers were taken when the
    rotary was made: another tensor under the name would not be seen, and the
    old one's memory would be read after it is freed."""
    rot = mcs.Rotary(64, axes=(12, 10, 10), magnitude=1.5, device="cpu")
    for name, value in (("turns", rot.turns.clone()), ("axis", rot.axis.clone()), ("magnitude", 2.0), ("layout", "interleaved"),
                        ("dims", 32), ("axes", (32,)), ("d", 128), ("_c", None)):
        before = getattr(rot, name)
        with pytest.raises(AttributeError):
            setattr(rot, name, value)
        assert getattr(rot, name) is before
        with pytest.raises(AttributeError):
            delattr(rot, name)
    assert rot._c.turns == rot.turns.data_ptr() and rot._c.axis == rot.axis.data_ptr()
    rot.label = "mine"                                    # (a name of the caller's own)
    assert copy.copy(rot).turns is rot.turns


def test_a_cache_keeps_its_buffers():
    cache = mcs.KVCache.empty(1, 1, 16, 64, page=16, device="cpu")
    with pytest.raises(AttributeError):
        del cache.page_table
    assert cache._c.page_table == cache.page_table.data_ptr()


# pi to 60 digits
PI = Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494"))


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0, layout="interleaved"), dict(axes=(22, 21, 21)),
                                dict(scaling=("linear", 3.0)), dict(scaling=("ntk", 7.0)), dict(base=1.01),
                                dict(scaling=("bands", 8.0, 1.0, 32.0, 8192)), dict(base=0.001), dict(base=1e30)])
def test_turns_are_the_nearest_fractions(kw):
    """round(f / 2 pi * 2^64) mod 2^64 of each frequency: off by half at most, so a
    position p's phase by |p| 2^-65 turns (in 53 bits it was off by hundreds)."""
    rot = mcs.Rotary(128, device="cpu", **kw)
    for f, turns in zip(rot.frequencies, rot.turns.tolist()):
        off = (Fraction(f) / (2 * PI) * 2 ** 64 - turns) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2) + Fraction(1, 10 ** 6)
