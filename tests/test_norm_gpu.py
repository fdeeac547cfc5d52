"""Norms and 8-bit rows on the GPU against their 64-bit forms."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref, rows_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def outputs(R, W, dtype, y=True, codes=True):
    """Outputs filled with what no test expects."""
    return (torch.full((R, W), 7.0, dtype=dtype, device=DEV) if y else None,
            torch.full((R, W), 7.0, device=DEV).to(F8) if codes else None,
            torch.full((R, -(-W // 128)), 7.0, device=DEV) if codes else None)


def check(got, want, units, dtype):
    y, codes, scales = got
    if y is not None:
        assert layer_ref.worst(y.cpu(), want, ref.norm_bound(want, units, dtype)) <= 1
    if codes is not None:
        ref.check_codes(codes.cpu(), scales.cpu(), want, units)


def up(t):
    return None if t is None else t.to(DEV)


# (R, H, D): heads within a wave of every width, whole rows and heads of other widths
# on both sides of each workgroup size, odd widths (one channel at a time), widths
# that end inside a block.
SHAPES = [(1, 1, 16), (5, 3, 16), (3, 7, 32), (2, 5, 64), (9, 4, 128), (3, 3, 256), (2, 2, 512),
          (1, 1, 128), (7, 1, 512), (1, 1, 8), (4, 1, 24), (3, 1, 504), (2, 3, 384), (5, 2, 640),
          (2, 1, 2048), (3, 1, 2056), (1, 1, 4096), (2, 1, 4104), (2, 1, 8192), (1, 1, 8200),
          (2, 1, 32768), (1, 2, 16384), (3, 1, 1), (2, 1, 7), (5, 1, 127), (2, 1, 129),
          (3, 1, 513), (2, 1, 1001), (2, 1, 4095), (1, 1, 4097), (2, 1, 32767)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,H,D", SHAPES)
def test_every_form(R, H, D, io):
    require_gpu()
    announce(f"norm R={R} H={H} D={D} io={io}")
    dtype, W = io_dtype(io), H * D
    gen = torch.Generator().manual_seed(R * 100000 + W)
    x = (torch.randn(R, W, generator=gen) * 3).to(dtype)
    gate = (torch.randn(R, W, generator=gen) * 3).to(dtype)
    weight = 1 + 0.3 * torch.randn(H, D, generator=gen)
    eps = 1e-5
    for form, use_weight, y_too, codes_too in [
            ("", True, True, True), ("", False, True, False), ("bf16", True, False, True),
            ("f32", True, True, True), ("after", True, False, True), ("before", True, True, True),
            ("before", False, True, False), ("after", False, True, True)]:
        res = (torch.randn(R, W, generator=gen) * 2).to(io_dtype(form)) if form in ("bf16", "f32") \
            else None
        g = gate if form in ("after", "before") else None
        w = weight if use_weight else None
        want, stored, units = ref.norm(x, w, eps, res, g, form == "before", H)
        got = outputs(R, W, dtype, y_too, codes_too)
        r = up(res)
        gdr.gdr_rms_norm(x.to(DEV), up(w), *got, residual=r, gate=up(g),
                         gate_first=form == "before", eps=eps, heads=H)
        check(got, want, units, dtype)
        if res is not None:
            bound = layer_ref.HALF[res.dtype] * stored.abs() + ref.U * stored.abs()
            assert layer_ref.worst(r.cpu(), stored, bound + 1e-37) <= 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("R,W", [(1, 1), (3, 128), (2, 100), (5, 4096), (2, 4111), (3, 65536),
                                 (1, 32760), (300, 256)])
def test_plain_rows(R, W, io):
    require_gpu()
    announce(f"quant R={R} W={W} io={io}")
    gen = torch.Generator().manual_seed(W)
    x = (torch.randn(R, W, generator=gen) * torch.exp(torch.randn(R, W, generator=gen))).to(
        io_dtype(io))
    _, codes, scales = outputs(R, W, x.dtype, y=False)
    gdr.gdr_quant_rows(x.to(DEV), codes, scales)
    ref.check_codes(codes.cpu(), scales.cpu(), x.double(), torch.zeros(R, W, dtype=ref.F64))
    as_bytes = torch.zeros(R, W, dtype=torch.uint8, device=DEV)
    gdr.gdr_quant_rows(x.to(DEV), as_bytes, scales)
    assert torch.equal(as_bytes, codes.view(torch.uint8))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("H,D", [(1, 1000), (3, 128), (5, 32), (1, 2500), (1, 333), (2, 384)])
@pytest.mark.parametrize("lo,width", [(0, 0), (8, 16), (3, 5), (0, 1)])
def test_slices_of_wider_rows(H, D, lo, width, io):
    """x and the gate as slices of a product's rows: aligned and unaligned starts and
    strides give the same digits as dense rows."""
    require_gpu()
    announce(f"norm slice H={H} D={D} lo={lo} pad={width} io={io}")
    R, W, dtype = 5, H * D, io_dtype(io)
    gen = torch.Generator().manual_seed(W + lo)
    rows = torch.randn(R, 2 * W + lo + width, generator=gen).to(dtype).to(DEV)
    x, gate = rows[:, lo: lo + W], rows[:, lo + W: lo + 2 * W]
    weight = torch.rand(H, D, generator=gen).to(DEV)
    for first in (False, True):
        want, _, units = ref.norm(x.cpu(), weight.cpu(), 1e-6, None, gate.cpu(), first, H)
        got, dense = outputs(R, W, dtype), outputs(R, W, dtype)
        gdr.gdr_rms_norm(x, weight, *got, gate=gate, gate_first=first)
        check(got, want, units, dtype)
        gdr.gdr_rms_norm(x.contiguous(), weight, *dense, gate=gate.contiguous(), gate_first=first)
        for a, b in zip(got, dense):
            assert torch.equal(a, b)
    off = torch.rand(W + 1, generator=gen).to(DEV)[1:].view(H, D)     # a weight off 16 bytes
    got = outputs(R, W, dtype)
    gdr.gdr_rms_norm(x, off, *got)
    check(got, *[t for i, t in enumerate(ref.norm(x.cpu(), off.cpu(), 1e-6, heads=H)) if i != 1],
          dtype)


@pytest.mark.parametrize("H,D", [(1, 2048), (4, 64), (1, 130), (2, 384), (1, 77)])
@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-19, 1e19, 1e30, 1e38])
def test_rows_of_any_magnitude(H, D, size):
    """Squares past fp32's range in either direction; eps of the rows' own size or less."""
    require_gpu()
    announce(f"norm H={H} D={D} size={size}")
    R, W = 3, H * D
    gen = torch.Generator().manual_seed(D)
    x = torch.randn(R, W, generator=gen).clamp(-3, 3) * size
    eps = 1e-37
    want, _, units = ref.norm(x, None, eps, heads=H)
    got = outputs(R, W, torch.float32)
    gdr.gdr_rms_norm(x.to(DEV), None, *got, eps=eps, heads=H)
    # Subnormal inputs keep fewer digits once eps has divided them; they are exact
    # before, and y is far above the smallest normal value unless x is subnormal.
    assert layer_ref.worst(got[0].cpu(), want, ref.norm_bound(want, units, torch.float32)
                           + (2.0 ** -126 if size < 1e-37 else 0)) <= 1


def test_rows_of_zeros_and_floors_of_the_scale():
    require_gpu()
    announce("norm of zeros, smallest scales")
    x = torch.zeros(2, 384)
    x[1, 128:256] = 1e-38
    got = outputs(2, 384, torch.float32)
    gdr.gdr_rms_norm(x.to(DEV), None, *got, eps=1e-6)
    assert (got[0][0] == 0).all() and (got[1][0].float() == 0).all()
    assert (got[2][0] == 2.0 ** -100).all()
    gdr.gdr_quant_rows(x.to(DEV), got[1], got[2])
    assert (got[2] == 2.0 ** -100).all()
    top = torch.full((1, 128), 3.0e38)
    _, codes, scales = outputs(1, 128, torch.float32, y=False)
    gdr.gdr_quant_rows(top.to(DEV), codes, scales)
    ref.check_codes(codes.cpu(), scales.cpu(), top.double(), torch.zeros(1, 128, dtype=ref.F64))


@pytest.mark.parametrize("W", [512, 640, 2500, 333])
def test_what_is_not_finite_stays_in_its_row(W):
    require_gpu()
    announce(f"norm and quant with inf and NaN W={W}")
    gen = torch.Generator().manual_seed(W)
    x = torch.randn(6, W, generator=gen)
    x[1, 3], x[3, W - 1], x[4, 130] = math.inf, math.nan, -math.inf
    want, _, units = ref.norm(x, None, 1e-6)
    got = outputs(6, W, torch.float32)
    gdr.gdr_rms_norm(x.to(DEV), None, *got)
    ok = [0, 2, 5]
    check([t[ok] for t in got], want[ok], units[ok], torch.float32)
    assert torch.isnan(got[0][3]).all() and torch.isnan(got[1][3].float()).all()
    # Plain rows: the scale is that of the finite values, infinities saturate.
    _, codes, scales = outputs(6, W, torch.float32, y=False)
    gdr.gdr_quant_rows(x.to(DEV), codes, scales)
    c, fine = codes.cpu().float(), torch.isfinite(x)
    y = torch.where(fine, x, 0.0).double()
    assert torch.isnan(c[3, W - 1]) and c[1, 3] == 448 and c[4, 130] == -448
    ref.check_codes(torch.where(fine, c, 0.0), scales.cpu(), y,
                    torch.zeros(6, W, dtype=ref.F64))


@pytest.mark.parametrize("R,H,D", [(1_200_000, 16, 16), (560_000, 1, 4096), (700_000, 8, 512)])
def test_many_rows(R, H, D):
    """More heads than workgroups, and tensors of more than 2^31 values."""
    require_gpu()
    announce(f"norm of many rows R={R} H={H} D={D}")
    W = H * D
    gen = torch.Generator(device=DEV).manual_seed(1)
    rows = torch.tensor([0, 1, R // 2, R - 2, R - 1], device=DEV)
    x = torch.zeros(R, W, dtype=torch.bfloat16, device=DEV)
    x[rows] = torch.randn(len(rows), W, generator=gen, device=DEV).bfloat16()
    w = torch.rand(H, D, generator=gen, device=DEV)
    y = torch.empty_like(x)
    codes = torch.empty(R, W, dtype=F8, device=DEV)
    scales = torch.empty(R, W // 128, device=DEV)
    gdr.gdr_rms_norm(x, w, y, codes, scales)
    want, _, units = ref.norm(x[rows].cpu(), w.cpu(), 1e-6, heads=H)
    check([t.view(torch.uint8)[rows].view(F8) if t.dtype == F8 else t[rows]
           for t in (y, codes, scales)], want, units, torch.bfloat16)
    y[rows] = 0
    assert not y.any() and (scales.min() == 2.0 ** -100).all()


def test_no_rows():
    require_gpu()
    announce("norm and quant of no rows")
    e = torch.empty(0, 256, device=DEV)
    gdr.gdr_rms_norm(e, None, torch.empty_like(e), heads=2)
    gdr.gdr_quant_rows(e, torch.empty(0, 256, dtype=F8, device=DEV), torch.empty(0, 2, device=DEV))


def test_refusals_of_the_binding():
    require_gpu()
    announce("norm refusals")
    z = lambda *s, **k: torch.zeros(*s, device=DEV, **k)  # noqa: E731
    x, y = z(4, 256), z(4, 256)
    codes, scales = z(4, 256).to(F8), z(4, 2)
    for kw in (dict(weight=z(255)), dict(weight=z(2, 64)), dict(weight=z(3, 100)), dict(heads=3),
               dict(weight=z(2, 128), heads=4), dict(residual=z(4, 255)), dict(gate=z(4, 255)),
               dict(gate=z(4, 256, dtype=torch.bfloat16)), dict(gate=z(256, 4).t()),
               dict(codes=codes), dict(scales=scales), dict(codes=codes, scales=z(4, 3)),
               dict(codes=z(4, 256), scales=scales), dict(residual=z(4, 256).half())):
        with pytest.raises((ValueError, TypeError)):
            gdr.gdr_rms_norm(x, y=y, **kw)
    for kw in (dict(residual=y), dict(y=x), dict(eps=0.0), dict(y=None),
               dict(residual=z(4, 256), gate=z(4, 256)), dict(heads=16 * 2)):
        with pytest.raises(gdr.GdrError):
            gdr.gdr_rms_norm(x, **{"y": y, **kw})
    with pytest.raises(ValueError):
        gdr.gdr_quant_rows(x[:, ::2], codes, scales)
    with pytest.raises(ValueError):
        gdr.gdr_quant_rows(x, None, scales)
    assert (y == 0).all() and (x == 0).all()
