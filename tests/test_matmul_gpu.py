"""The 8-bit product on the GPU against its 64-bit form."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref, rows_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def inputs(seed, M, N, K, bias=True):
    """Codes of every size and any scales, on the GPU."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    kb, nb = -(-K // 128), -(-N // 128)
    return ((r(M, K) * 40).clamp(-448, 448).to(F8), torch.exp(r(M, kb) * 2) * 0.01,
            (r(N, K) * 40).clamp(-448, 448).to(F8), torch.exp(r(nb, kb) * 2) * 0.01,
            r(N) * 30 if bias else None)


def run(x, sx, w, sw, bias, dtype):
    y = torch.full((x.shape[0], w.shape[0]), 7.0, dtype=dtype, device=DEV)
    gdr.gdr_matmul_fp8(x, sx, w, sw, y, bias=bias)
    return y


def check(args, dtype):
    y = run(*args, dtype)
    x, sx, w, sw, bias = args
    want, mag = ref.matmul(x.double(), sx, w.double(), sw, bias)   # 64-bit on the GPU
    worst = layer_ref.worst(y, want, ref.matmul_bound(want, mag, dtype, x.shape[1]))
    assert worst <= 1, worst
    # On the whole a partial sum is no larger than the result: half of two units at each
    # addition of a block, and a rounding at each of the sum over blocks.
    # The 8-bit instructions' truncation (2^-13 of the largest of 8 products, half of that
    # on average, each) is far below bf16's rounding (at most 2^-8, 2^-9 on average).
    if want.numel() > 1000:
        rel = layer_ref.rel(y, want)
        most = (128 + x.shape[1] // 128 + 4) * ref.U if dtype == torch.float32 else 2.0 ** -9
        assert rel < most, (rel, most)
    return y


# (M, N, K): one row, both sides of every tile's edge, outputs that are not of whole
# vectors or blocks, channels that end inside a block or a lane's 32.
SHAPES = [(1, 1, 16), (1, 4, 128), (1, 128, 144), (1, 1000, 4096), (3, 5, 48), (16, 16, 128),
          (17, 33, 160), (15, 130, 1040), (31, 64, 256), (32, 96, 2048), (33, 200, 272),
          (64, 256, 1024), (65, 255, 1008), (100, 129, 384), (128, 128, 128), (129, 257, 256),
          (200, 1003, 2064), (255, 513, 528), (256, 256, 4096), (257, 768, 640), (300, 2048, 512),
          (513, 1024, 1040), (1000, 516, 2048), (700, 3000, 768)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K, io):
    require_gpu()
    announce(f"matmul M={M} N={N} K={K} io={io}")
    for bias in (True, False):
        check(inputs(M + N + K, M, N, K, bias), io_dtype(io))


# Sizes that take each of the kernel's tilings, with whole and with ragged tiles.
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(16, 272, 1168), (32, 300, 656), (64, 8192, 272),
                                   (100, 8192, 272), (97, 8184, 656), (192, 8192, 400),
                                   (201, 8001, 144), (512, 8192, 272), (500, 8100, 528),
                                   (1000, 8192, 272), (990, 8190, 400), (1536, 8192, 400),
                                   (1500, 8001, 272), (1500, 8008, 1296)])
def test_every_tiling(M, N, K, io):
    require_gpu()
    announce(f"matmul tiling M={M} N={N} K={K} io={io}")
    check(inputs(M + N, M, N, K), io_dtype(io))


# The tilings of few rows, or of few outputs for the rows there are; blocks enough that
# each of their waves takes several.
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(7, 300, 2064), (8, 1003, 4112), (8, 8192, 2048), (9, 300, 4112),
                                   (20, 1000, 1040), (45, 2001, 2064), (48, 4096, 1296),
                                   (33, 4100, 2064), (64, 4099, 1040), (100, 2003, 4112),
                                   (200, 1003, 4000), (250, 4001, 1040), (60, 16003, 1296),
                                   (500, 8100, 2064), (990, 8190, 1040), (1500, 8001, 2064)])
def test_tilings_of_few_rows_or_outputs(M, N, K, io):
    require_gpu()
    announce(f"matmul tiling of few M={M} N={N} K={K} io={io}")
    check(inputs(M + N, M, N, K), io_dtype(io))


# Rows a multiple of 4 KiB or 512 bytes apart, whose workgroups begin at different blocks.
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 8192, 4096), (5, 6000, 8192), (16, 1600, 4096),
                                   (30, 5003, 4096), (40, 4100, 12288), (64, 8192, 4096),
                                   (61, 16003, 4096), (130, 2001, 8192), (250, 1000, 4096),
                                   (400, 5003, 4608), (1000, 8190, 8704), (1100, 8001, 4608),
                                   (1500, 8001, 8704), (1536, 8192, 12288), (700, 8100, 17408)])
def test_rows_of_whole_pages(M, N, K, io):
    require_gpu()
    announce(f"matmul rows of whole pages M={M} N={N} K={K} io={io}")
    check(inputs(M + N, M, N, K), io_dtype(io))


@pytest.mark.parametrize("M,N,K", [(4000, 8192, 4096), (2047, 4100, 1040), (1, 8192, 14336),
                                   (64, 4096, 14336), (4097, 128, 4096), (5000, 16, 256),
                                   (16, 20000, 512)])
def test_large_products(M, N, K):
    require_gpu()
    announce(f"matmul M={M} N={N} K={K}")
    check(inputs(7, M, N, K), torch.bfloat16)


def test_weights_past_32_bits_of_bytes():
    """Offsets of the last rows of a weight of over 4 GiB."""
    require_gpu()
    announce("matmul over a weight of 4.3 GiB")
    N, K = 70000, 65536
    gen = torch.Generator(device=DEV).manual_seed(3)
    w = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    rows = torch.tensor([0, 1, 32767, 32768, 65535, 65536, N - 1], device=DEV)
    w[rows] = (torch.randn(len(rows), K, generator=gen, device=DEV) * 40).to(F8).view(torch.uint8)
    sw = torch.rand(-(-N // 128), K // 128, generator=gen, device=DEV)
    for M in (3, 300):
        x = (torch.randn(M, K, generator=gen, device=DEV) * 40).to(F8)
        sx = torch.rand(M, K // 128, generator=gen, device=DEV) * 0.01
        y = torch.empty(M, N, device=DEV)
        gdr.gdr_matmul_fp8(x, sx, w.view(F8), sw, y)
        a = x.double() * ref.spread(sx.double(), K)
        b = w[rows].view(F8).double() * ref.spread(sw.double()[rows // 128], K)
        want, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
        assert layer_ref.worst(y[:, rows], want,
                               ref.matmul_bound(want, mag, torch.float32, K)) <= 1
        y[:, rows] = 0
        assert (y == 0).all()


@pytest.mark.parametrize("M", [5, 40, 300])
def test_exact_where_every_sum_is(M):
    """Small whole codes and power-of-two scales: no rounding anywhere."""
    require_gpu()
    announce(f"matmul exact M={M}")
    gen = torch.Generator(device=DEV).manual_seed(M)
    N, K = 300, 400
    x = torch.randint(-3, 4, (M, K), generator=gen, device=DEV).float().to(F8)
    w = torch.randint(-3, 4, (N, K), generator=gen, device=DEV).float().to(F8)
    sx = 2.0 ** torch.randint(-3, 3, (M, 4), generator=gen, device=DEV)
    sw = 2.0 ** torch.randint(-3, 3, (3, 4), generator=gen, device=DEV)
    bias = torch.randint(-9, 9, (N,), generator=gen, device=DEV).float()
    y = run(x, sx, w, sw, bias, torch.float32)
    want, _ = ref.matmul(x.double(), sx, w.double(), sw, bias)
    assert torch.equal(y.double(), want)
    # Codes of the subnormal range and the largest ones.
    tiny = torch.full((M, K), 2.0 ** -9, device=DEV).to(F8)
    y = run(tiny, torch.ones_like(sx), torch.full((N, K), 448.0, device=DEV).to(F8),
            torch.ones_like(sw), None, torch.float32)
    assert (y == K * 448 * 2.0 ** -9).all()


@pytest.mark.parametrize("M,N,K", [(5, 40, 272), (40, 130, 1040), (300, 300, 400)])
def test_what_is_not_finite_stays_in_its_row_and_column(M, N, K):
    """NaN codes and scales that are not finite reach what depends on them alone, also
    next to the ends of rows, columns and channels."""
    require_gpu()
    announce(f"matmul with NaN M={M} N={N} K={K}")
    x, sx, w, sw, bias = inputs(1, M, N, K)
    want, mag = ref.matmul(x.double(), sx, w.double(), sw, bias)
    x8, w8 = x.view(torch.uint8), w.view(torch.uint8)
    x8[M - 1, K - 1] = 0x7f
    x8[0, 0] = 0xff
    w8[N - 1, K - 1] = 0xff
    w8[1, 17] = 0x7f
    sx[2, 0] = math.inf
    bias[3] = math.nan
    y = run(x, sx, w, sw, bias, torch.float32)
    assert torch.isnan(y[[0, M - 1]]).all() and torch.isnan(y[:, [1, 3, N - 1]]).all()
    assert not torch.isfinite(y[2]).any()
    rows = [i for i in range(M) if i not in (0, 2, M - 1)]
    cols = [i for i in range(N) if i not in (1, 3, N - 1)]
    bound = ref.matmul_bound(want, mag, torch.float32, K)
    pick = lambda t: t[rows][:, cols]  # noqa: E731
    assert layer_ref.worst(pick(y), pick(want), pick(bound)) <= 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_no_channels_rows_or_outputs(io):
    require_gpu()
    announce("matmul of nothing")
    dtype = io_dtype(io)
    for M, N in ((3, 5), (200, 130), (1, 1)):
        x, sx = torch.empty(M, 0, device=DEV).to(F8), torch.empty(M, 0, device=DEV)
        w, sw = torch.empty(N, 0, device=DEV).to(F8), torch.empty(-(-N // 128), 0, device=DEV)
        bias = torch.randn(N, device=DEV)
        assert (run(x, sx, w, sw, None, dtype) == 0).all()
        assert torch.equal(run(x, sx, w, sw, bias, dtype), bias.to(dtype).expand(M, N))
    x, sx, w, sw, _ = inputs(1, 4, 8, 128)
    run(x[:0], sx[:0], w, sw, None, dtype)
    run(x, sx, w[:0], sw[:0], None, dtype)


@pytest.mark.parametrize("M", [2, 50, 200, 600])
def test_same_digits_every_time(M):
    require_gpu()
    announce(f"matmul repeated M={M}")
    args = inputs(9, M, 520, 2000)
    first = run(*args, torch.float32)
    for _ in range(4):
        assert torch.equal(run(*args, torch.float32), first)


def test_refusals_of_the_binding():
    require_gpu()
    announce("matmul refusals")
    x, sx, w, sw, bias = inputs(1, 4, 130, 272)
    y = torch.zeros(4, 130, device=DEV)
    f = torch.zeros(4, 272, device=DEV)
    for args in ((f, sx, w, sw, y), (x, sx, f, sw, y), (x, sx[:, :2].contiguous(), w, sw, y),
                 (x, sx, w, sw[:1].contiguous(), y), (x, sx, w, sw, y[:, :129].contiguous()),
                 (x, sx, w[:, :256].contiguous(), sw, y), (x.t(), sx, w, sw, y),
                 (x, sx.double(), w, sw, y), (x, sx, w, sw, y.half())):
        with pytest.raises((ValueError, TypeError)):
            gdr.gdr_matmul_fp8(*args)
    with pytest.raises(ValueError):
        gdr.gdr_matmul_fp8(x, sx, w, sw, y, bias=bias[:5])
    with pytest.raises(gdr.GdrError):                       # K not a multiple of 16
        gdr.gdr_matmul_fp8(x[:, :264].contiguous(), sx, w[:, :264].contiguous(), sw, y)
    assert (y == 0).all()
