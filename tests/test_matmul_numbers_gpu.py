"""Numbers of the 8-bit product, in all tilings and both output types: exact where every
sum is, the same digits every time, outliers that cancel, and scales of every size."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref, rows_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn

# Each tiling, with rows that lie a multiple of 4 KiB or of 512 bytes apart (whose workgroups
# begin at different blocks) and others, whole and ragged tiles.
SHAPES = [(3, 300, 4096), (3, 300, 2064), (16, 1000, 4096), (8, 8200, 8192), (30, 1003, 4096),
          (24, 4100, 8192), (48, 2001, 4096), (48, 2001, 1296), (33, 4096, 12288), (40, 4100, 4096),
          (64, 8192, 4096), (64, 4096, 14336), (61, 16003, 4096), (60, 16000, 1296),
          (100, 5003, 4096), (128, 2001, 8192), (192, 8192, 4608), (201, 8001, 400),
          (300, 8192, 4608), (512, 8192, 8704), (500, 8100, 528), (640, 8190, 4096),
          (1000, 8192, 8704), (990, 8190, 656), (1100, 8001, 4608), (1536, 8192, 4608),
          (1500, 8001, 4096), (1500, 8008, 1296)]


def call(x, sx, w, sw, bias, dtype):
    y = torch.full((x.shape[0], w.shape[0]), 7.0, dtype=dtype, device=DEV)
    gdr.gdr_matmul_fp8(x, sx, w, sw, y, bias=bias)
    return y


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers_round_once(M, N, K, io):
    """Codes from -3 to 3, scales of 1 and 2 and a whole bias: products are at most 9, sums
    whole and below 2^24, so that any order of either kind of instruction is exact and the
    output is the sum's one rounding, value for value."""
    require_gpu()
    announce(f"matmul of whole numbers M={M} N={N} K={K} io={io}")
    assert 4 * 9 * K + 9 < 2 ** 24
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device=DEV).float()  # noqa: E731
    kb, nb = -(-K // 128), -(-N // 128)
    x, w, sx, sw = r(-3, 4, M, K).to(F8), r(-3, 4, N, K).to(F8), r(1, 3, M, kb), r(1, 3, nb, kb)
    bias = r(-9, 10, N)
    want, _ = ref.matmul(x.double(), sx, w.double(), sw, bias)
    y = call(x, sx, w, sw, bias, io_dtype(io))
    assert torch.equal(y, want.to(y.dtype))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_same_digits_every_time(M, N, K, io):
    require_gpu()
    announce(f"matmul repeated M={M} N={N} K={K} io={io}")
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    kb, nb = -(-K // 128), -(-N // 128)
    args = [(r(M, K) * 40).clamp(-448, 448).to(F8), torch.exp(r(M, kb)),
            (r(N, K) * 40).clamp(-448, 448).to(F8), torch.exp(r(nb, kb)), r(N)]
    first = call(*args, io_dtype(io))
    assert torch.isfinite(first).all()
    other = torch.empty(N, M, dtype=first.dtype, device=DEV)
    for _ in range(4):
        gdr.gdr_matmul_fp8(args[2], torch.ones(N, kb, device=DEV), args[0],
                           torch.ones(-(-M // 128), kb, device=DEV), other)
        assert torch.equal(call(*args, io_dtype(io)), first)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(5, 320), (40, 320), (100, 5000), (600, 8200), (1500, 8192)])
def test_outliers_that_cancel(M, N, io):
    """One product of every eight neighbours is the largest there is, and the next eight's is
    its negative: what is left is the small ones' sum, to 2^-10 of the terms' magnitudes in
    bf16 and to fp32's roundings in fp32."""
    require_gpu()
    announce(f"matmul with outliers M={M} N={N} io={io}")
    K = 1024
    gen = torch.Generator(device=DEV).manual_seed(M)
    x, w = (torch.randn(n, K, generator=gen, device=DEV) for n in (M, N))
    x[:, ::8], w[:, ::16], w[:, 8::16] = 448, 448, -448
    x, w = x.to(F8), w.to(F8)
    sx, sw = torch.ones(M, 8, device=DEV), torch.ones(-(-N // 128), 8, device=DEV)
    want, mag = ref.matmul(x.double(), sx, w.double(), sw)
    assert (want.abs().amax() < 2.0 ** -10 * mag.amin()).all()
    y = call(x, sx, w, sw, None, io_dtype(io))
    assert layer_ref.worst(y, want, ref.matmul_bound(want, mag, y.dtype, K)) <= 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(5, 320), (40, 320), (100, 5000), (600, 8200), (1500, 8192)])
def test_scales_of_every_size(M, N, io):
    """Scales far from 1 whose products are normal numbers, large ones on blocks of zeros
    among them; where a product of scales is past fp32's range (row 2, the first 128
    outputs), nothing else changes."""
    require_gpu()
    announce(f"matmul with scales of every size M={M} N={N} io={io}")
    K = 1008
    gen = torch.Generator(device=DEV).manual_seed(N)
    rand = lambda *s: 1 + torch.rand(*s, generator=gen, device=DEV)  # noqa: E731
    x, w = ((torch.randn(n, K, generator=gen, device=DEV) * 40).clamp(-448, 448).to(F8)
            for n in (M, N))
    x.view(torch.uint8)[:, 384: 512] = 0
    up = torch.tensor([100, -100, 60, 100, -126, 126, 0, -20], device=DEV)
    down = torch.tensor([-100, 100, -58, 25, 126, -126, 0, 20], device=DEV)
    sx, sw = rand(M, 8) * 2.0 ** up, rand(-(-N // 128), 8) * 2.0 ** down
    for tiny in (False, True):
        if tiny:                          # the smallest normal products, of the scales' floor
            sx[:], sw[:] = 2.0 ** -100 * rand(M, 8), 2.0 ** -26 * rand(-(-N // 128), 8)
        want, mag = ref.matmul(x.double(), sx, w.double(), sw)
        y = call(x, sx, w, sw, None, io_dtype(io))
        assert layer_ref.worst(y, want, ref.matmul_bound(want, mag, y.dtype, K)) <= 1
    sx[2, 3], sw[0, 3] = 2.0 ** 100, 2.0 ** 100
    again = call(x, sx, w, sw, None, io_dtype(io))
    rows = torch.arange(M, device=DEV) != 2
    assert not torch.isfinite(again[2, :128]).any()
    assert torch.equal(again[rows], y[rows]) and torch.equal(again[2, 128:], y[2, 128:])
