"""Norms of heads that hold an infinity, by the definition: h / sqrt(mean h^2 + eps) is
0 for the head's finite channels and NaN for its infinite ones; other heads and rows are
as without it."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref, rows_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu


def up(t):
    return None if t is None else t.to(DEV)


# Heads within a wave, heads and rows of a workgroup each (one vector a thread and more),
# widths that end inside a vector.
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["", "weight", "res", "after", "before"])
@pytest.mark.parametrize("H,D", [(5, 16), (3, 128), (2, 512), (2, 384), (1, 640), (1, 333),
                                 (1, 5000), (1, 20000)])
def test_heads_with_an_infinity(H, D, form, io):
    require_gpu()
    announce(f"norm with infinities H={H} D={D} {form} io={io}")
    dtype, R, W = io_dtype(io), 5, H * D
    gen = torch.Generator().manual_seed(W)
    x = torch.randn(R, W, generator=gen).to(dtype)
    x[1, 3], x[3, W - 1], x[4, 0], x[4, W // 2] = math.inf, -math.inf, math.inf, -math.inf
    weight = 1 + 0.3 * torch.randn(H, D, generator=gen) if form == "weight" else None
    res = torch.randn(R, W, generator=gen).to(dtype) if form == "res" else None
    gate = torch.randn(R, W, generator=gen).to(dtype) if form in ("after", "before") else None
    first = form == "before"
    want, stored, units = ref.norm(x, weight, 1e-6, res, gate, first, H)
    y, r = torch.full((R, W), 7.0, dtype=dtype, device=DEV), up(res)
    codes = torch.zeros(R, W, device=DEV).to(torch.float8_e4m3fn)
    scales = torch.full((R, -(-W // 128)), 7.0, device=DEV)
    gdr.gdr_rms_norm(up(x), up(weight), y, codes, scales, residual=r, gate=up(gate),
                     gate_first=first, heads=H)
    bad = torch.isnan(want)
    assert torch.equal(bad, torch.isinf(x)) and (want[1, :3] == 0).all()
    y, codes = y.cpu(), codes.cpu().float()
    assert torch.equal(torch.isnan(y), bad) and torch.equal(torch.isnan(codes), bad)
    want, y, codes = (torch.where(bad, 0, t) for t in (want, y, codes))
    assert layer_ref.worst(y, want, ref.norm_bound(want, units, dtype)) <= 1
    ref.check_codes(codes, scales.cpu(), want, units)
    if res is not None:
        assert torch.equal(torch.isinf(r.cpu()), torch.isinf(stored))


def test_a_sum_past_the_range_of_fp32():
    """x + residual past fp32's range is infinite, and so is what is stored of it."""
    require_gpu()
    announce("norm of sums past fp32's range")
    x, r = torch.full((2, 256), 1.0), torch.full((2, 256), 1.0)
    x[0, 7] = r[0, 7] = 3e38
    y, r = torch.zeros(2, 256, device=DEV), r.to(DEV)
    gdr.gdr_rms_norm(x.to(DEV), None, y, residual=r)
    y, r = y.cpu(), r.cpu()
    assert torch.isinf(r[0, 7]) and torch.isnan(y[0, 7])
    r[0, 7], y[0, 7] = 2, 0
    assert (r == 2).all() and (y[0] == 0).all() and (y[1] - 1).abs().max() < 1e-6
