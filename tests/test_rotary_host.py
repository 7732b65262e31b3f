"""Rotary's tables on the host: the library holds their addresses, so they cannot
be rebound."""
import copy

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
