"""Plain 64-bit forms of the norms, the 8-bit product and the rotary positions, and
the bounds their kernels are held to (units are 2^-24, half a step of fp32)."""
from __future__ import annotations

import math

import torch

from tests.layer_ref import F64, HALF, clip_lens

U = 2.0 ** -24
BLOCK = 128


def silu(z):
    return z / (1 + torch.exp(-z))


def norm(x, weight, eps, residual=None, gate=None, gate_first=False, heads=1):
    """x [R,H*D] -> y, h (what the residual becomes) and the units y is off by."""
    R, W = x.shape
    h = x.to(F64)
    z = torch.zeros(R, W, dtype=F64) if gate is None else gate.to(F64)
    # silu: the rounding of the exponent's product and six more, and the product with it.
    gate_units = torch.zeros(R, W, dtype=F64) if gate is None else 1.5 * z.abs() + 8
    if residual is not None:
        h = h + residual.to(F64)
    stored = h
    if gate is not None and gate_first:
        h = h * silu(z)
    head = h.view(R, heads, W // heads)
    y = head / torch.sqrt((head * head).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.to(F64).view(heads, W // heads)
    y = y.reshape(R, W)
    # h itself (also by way of the root), the root's factor, two products and the weight's.
    units = 6 + gate_units
    if gate is not None and gate_first:
        units = units + gate_units.view(R, heads, -1).amax(-1, keepdim=True).expand(
            R, heads, W // heads).reshape(R, W)
    elif gate is not None:
        y = y * silu(z)
    return y, stored, units


def norm_bound(y, units, dtype):
    return HALF[dtype] * y.abs() + units * U * y.abs() + 1e-36


def blocks(t):
    n = -(-t.shape[-1] // BLOCK)
    t = torch.nn.functional.pad(t, (0, n * BLOCK - t.shape[-1]))
    return t.view(*t.shape[:-1], n, BLOCK)


def scales(y):
    return (blocks(torch.where(torch.isfinite(y), y, 0.0)).abs().amax(-1) / 448).clamp(
        min=2.0 ** -100)


def spread(s, width):
    return s.repeat_interleave(BLOCK, -1)[..., :width]


def check_codes(codes, got_scales, y, units):
    """Codes and scales against the finite y they stand for, `units` off at most."""
    want = scales(y)
    most = spread(blocks(units).amax(-1), y.shape[-1])
    s = got_scales.to(F64)
    # The scale: the largest value's error, and one product.
    assert ((s - want).abs() <= want * (blocks(most).amax(-1) + 2) * U).all()
    s = spread(s, y.shape[-1])
    # A code: half a step (2^-4 of a normal value, 2^-10 of a subnormal one), the
    # value's own error, the inverse's and the product's.
    bound = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) + (units + 3) * U * y.abs()
    assert ((codes.to(F64) * s - y).abs() <= bound).all()


def matmul(x, sx, w, sw, bias=None):
    """Values of codes x [M,K], w [N,K] -> y and the sum of its terms' magnitudes."""
    K, N = x.shape[1], w.shape[0]
    a = x.to(F64) * spread(sx.to(F64), K)
    b = w.to(F64) * spread(sw.to(F64).repeat_interleave(BLOCK, 0)[:N], K)
    b, ab = b.t().contiguous(), b.abs().t().contiguous()
    y, mag = a @ b, a.abs() @ ab
    if bias is not None:
        y, mag = y + bias.to(F64), mag + bias.to(F64).abs()
    return y, mag


def matmul_bound(y, mag, dtype, K):
    # fp32: a block's 128 products are exact and its sum rounds (or truncates: two
    # units) at each addition; then two scales, one multiply-add a block, and the bias.
    units = 2 * BLOCK + -(-K // BLOCK) + 16
    bound = HALF[dtype] * y.abs() + units * U * mag + 1e-36
    # bf16: of 8 products each loses less than 2^-13 of the largest, so a group loses
    # less than 8 2^-13 of its terms' magnitudes.
    return bound if dtype == torch.float32 else bound + 2.0 ** -10 * mag


def rope(x, freq, pos, Hq, Hkv, D, interleaved, magnitude, lens=None, fill=0.0):
    """x [B,T,heads*D] -> all heads turned, and a bound of each value's magnitude."""
    B, T = x.shape[:2]
    R = 2 * freq.shape[0]
    heads = x.shape[2] // D
    t = x.to(F64).view(B, T, heads, D)
    p = pos.to(torch.int64)[:, None] + torch.arange(T)
    angle = p[..., None].to(F64) * freq
    c, s = torch.cos(angle)[:, :, None] * magnitude, torch.sin(angle)[:, :, None] * magnitude
    y, mag = t.clone(), torch.zeros_like(t)
    one = slice(0, R, 2) if interleaved else slice(0, R // 2)
    two = slice(1, R, 2) if interleaved else slice(R // 2, R)
    n = Hq + Hkv
    a, b = t[:, :, :n, one], t[:, :, :n, two]
    y[:, :, :n, one], y[:, :, :n, two] = a * c - b * s, a * s + b * c
    mag[:, :, :n, one] = mag[:, :, :n, two] = (a.abs() + b.abs()) * abs(magnitude)
    for i, k in enumerate(clip_lens(lens, B, T)):
        y[i, k:], mag[i, k:] = fill, 0
    return y, mag


def rope_bound(y, mag, dtype, pos=0):
    # The turn's fraction rounds to fp32 (2 pi 2^-26), sine and cosine are off by two
    # units of themselves and their magnitude by one, each product and the sum by one;
    # the 64-bit turns are off by two of their own roundings.
    turns = 2 * math.pi * 2.0 ** -52 * (abs(pos) + 2.0 ** 12)
    return HALF[dtype] * torch.where(mag > 0, y.abs(), 0.0) + (8 * U + turns) * mag
