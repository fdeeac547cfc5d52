"""Frequencies of the rotary positions on the host, whatever device tensors are made on."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_40_amd as gdr


def test_frequencies_are_on_the_cpu_whatever_the_default_device():
    want, m = gdr.gdr_rope_freqs(64, 10000.0, kind=gdr.GDR_ROPE_LINEAR, factor=2.0)
    with torch.device("meta"):
        got, n = gdr.gdr_rope_freqs(64, 10000.0, kind=gdr.GDR_ROPE_LINEAR, factor=2.0)
    assert got.device.type == "cpu" and n == m and torch.equal(got, want)
    try:
        torch.set_default_device("meta")
        got, _ = gdr.gdr_rope_freqs(64, 10000.0)
    finally:
        torch.set_default_device(None)
    assert got.device.type == "cpu" and got[0] == 1.0


@pytest.mark.parametrize("R,base,factor", [(4, 1e4, 1e160), (128, 1e300, 1e10), (6, 1e5, 1e308)])
def test_a_larger_base_past_the_range_is_refused(R, base, factor):
    """It would be infinite, and every frequency but the first 0."""
    with pytest.raises(gdr.GdrError) as e:
        gdr.gdr_rope_freqs(R, base, kind=gdr.GDR_ROPE_BASE, factor=factor)
    assert e.value.status == -4
    f, _ = gdr.gdr_rope_freqs(R, base, kind=gdr.GDR_ROPE_BASE, factor=4.0)
    assert (f > 0).all()
