"""Sizes of the rotation's table (CPU)."""
import pytest

import paged_kv_cache_476_b200 as pkv


@pytest.mark.parametrize("positions,rot", [(16, 33), (16, -2), (0, 32)])
def test_refused(positions, rot):
    """(an odd rotary_dim lost a column, and with it every later angle)"""
    with pytest.raises(ValueError):
        pkv.rope_cos_sin(positions, rot, device="cpu")


@pytest.mark.parametrize("rot", [0, 2, 32, 128])
def test_taken(rot):
    assert pkv.rope_cos_sin(16, rot, device="cpu").shape == (16, rot)
