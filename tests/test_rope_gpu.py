"""Rotary positions on the GPU against their 64-bit form."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref, rows_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu


def run(x, freq, pos, Hq, Hkv, D, interleaved, magnitude=1.0, lens=None, with_v=True):
    """q, k, v side by side as [B,T,heads,D]; 7 where nothing was written."""
    B, T = x.shape[:2]
    out = [torch.full((B, T, h, D), 7.0, dtype=x.dtype, device=DEV) for h in (Hq, Hkv, Hkv)]
    gdr.gdr_rope(x, freq.to(DEV), pos.to(DEV), out[0], out[1], out[2] if with_v else None,
                 interleaved=interleaved, magnitude=magnitude,
                 lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV))
    return torch.cat(out if with_v else out[:2], 2)


def freqs(R, base=10000.0):
    return base ** (-2 * torch.arange(R // 2, dtype=torch.float64) / R) if R else \
        torch.empty(0, dtype=torch.float64)


# (D, R): whole heads, parts of them, nothing, pairs that fill 16 bytes or not
HEADS = [(64, 64), (128, 128), (256, 256), (512, 512), (8, 8), (8, 2), (128, 64), (128, 32),
         (64, 16), (64, 58), (128, 24), (40, 20), (64, 0), (96, 96), (256, 250), (72, 4)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", HEADS)
def test_heads(D, R, interleaved, io):
    require_gpu()
    announce(f"rope D={D} R={R} interleaved={interleaved} io={io}")
    for B, T, Hq, Hkv, lens in [(1, 1, 1, 1, None), (3, 1, 5, 2, [1, 0, 1]), (2, 37, 4, 1, [37, 20]),
                                (3, 9, 2, 2, [-1, 30, 5]), (1, 130, 3, 1, None)]:
        gen = torch.Generator().manual_seed(D + R + T)
        x = torch.randn(B, T, (Hq + 2 * Hkv) * D, generator=gen).to(io_dtype(io))
        pos = torch.randint(0, 5000, (B,), generator=gen).to(torch.int32)
        got = run(x.to(DEV), freqs(R), pos, Hq, Hkv, D, interleaved, 1.25, lens).cpu()
        want, mag = ref.rope(x, freqs(R), pos, Hq, Hkv, D, interleaved, 1.25, lens, fill=7.0)
        assert layer_ref.worst(got, want, ref.rope_bound(want, mag, x.dtype) + 1e-37) <= 1
        still = mag == 0                                    # copied, or behind the end
        assert torch.equal(got[still].double(), want[still])


@pytest.mark.parametrize("pos", [0, 1, 4095, 1000003, 2 ** 24 - 3, 2 ** 31 - 40, -5])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(pos, interleaved):
    require_gpu()
    announce(f"rope at {pos} interleaved={interleaved}")
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(1, 60, 4 * 64, generator=gen)
    p = torch.tensor([pos], dtype=torch.int32)              # the last tokens pass 2^31
    f, m = gdr.gdr_rope_freqs(64, 500000.0, kind=gdr.GDR_ROPE_INDEX, factor=32.0, context=32768.0,
                              low=1.0, high=32.0)
    got = run(x.to(DEV), f, p, 2, 1, 64, interleaved, m).cpu()
    want, mag = ref.rope(x, f, p, 2, 1, 64, interleaved, m)
    assert layer_ref.worst(got, want, ref.rope_bound(want, mag, x.dtype, pos) + 1e-37) <= 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lo,width", [(0, 0), (16, 32), (3, 5), (0, 1), (8, 12)])
def test_slices_of_wider_rows(lo, width, io):
    require_gpu()
    announce(f"rope slice lo={lo} pad={width} io={io}")
    B, T, Hq, Hkv, D = 2, 11, 3, 1, 64
    C = (Hq + 2 * Hkv) * D
    gen = torch.Generator().manual_seed(lo)
    rows = torch.randn(B, T, C + lo + width, generator=gen).to(io_dtype(io)).to(DEV)
    pos = torch.tensor([3, 900], dtype=torch.int32)
    for interleaved in (False, True):
        x = rows[:, :, lo: lo + C]
        got = run(x, freqs(48), pos, Hq, Hkv, D, interleaved)
        assert torch.equal(got, run(x.contiguous(), freqs(48), pos, Hq, Hkv, D, interleaved))
        one = run(rows[:, 4:5, lo: lo + C], freqs(48), pos + 4, Hq, Hkv, D, interleaved)
        assert torch.equal(one, got[:, 4:5])                # single tokens, rows far apart
        qk = run(rows[:, :, lo: lo + C - Hkv * D], freqs(48), pos, Hq, Hkv, D, interleaved,
                 with_v=False)
        assert torch.equal(qk, got[:, :, : Hq + Hkv])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (32, 8), (1, 3), (64, 64)])
def test_steps_equal_a_prompt(Hq, Hkv):
    require_gpu()
    announce(f"rope steps Hq={Hq} Hkv={Hkv}")
    D, T = 128, 20
    gen = torch.Generator().manual_seed(Hq)
    x = torch.randn(2, T, (Hq + 2 * Hkv) * D, generator=gen).to(torch.bfloat16).to(DEV)
    pos = torch.tensor([70, 0], dtype=torch.int32)
    whole = run(x, freqs(D), pos, Hq, Hkv, D, False)
    for t in (0, 1, 13, T - 1):
        assert torch.equal(run(x[:, t:t + 1], freqs(D), pos + t, Hq, Hkv, D, False),
                           whole[:, t:t + 1])


def test_many_tokens():
    """Rows of more than 2^31 values."""
    require_gpu()
    announce("rope of 540000 tokens")
    T, D = 540_000, 128
    gen = torch.Generator(device=DEV).manual_seed(2)
    rows = torch.tensor([0, 7, T // 2, T - 1], device=DEV)
    x = torch.zeros(1, T, 32 * D, dtype=torch.bfloat16, device=DEV)
    x[0, rows] = torch.randn(len(rows), 32 * D, generator=gen, device=DEV).bfloat16()
    pos = torch.tensor([5], dtype=torch.int32)
    got = run(x, freqs(D), pos, 24, 4, D, False)
    for r in rows.tolist():
        want, mag = ref.rope(x[:, r:r + 1].cpu(), freqs(D), pos + r, 24, 4, D, False, 1.0)
        assert layer_ref.worst(got[:, r:r + 1].cpu(), want,
                               ref.rope_bound(want, mag, x.dtype, 5 + r) + 1e-37) <= 1
    got[0, rows] = 0
    assert not got.any()


def test_what_is_not_finite_stays_in_its_pair():
    require_gpu()
    announce("rope with inf and NaN")
    x = torch.ones(1, 3, 4 * 64)
    x[0, 1, 5], x[0, 2, 64 + 40], x[0, 0, 3 * 64] = math.nan, math.inf, math.nan
    pos = torch.tensor([9], dtype=torch.int32)
    got = run(x.to(DEV), freqs(64), pos, 2, 1, 64, False).cpu()
    bad = ~torch.isfinite(got)
    at = {(1, 0, 5), (1, 0, 37), (2, 1, 40), (2, 1, 8), (0, 3, 0)}
    assert {tuple(i.tolist()) for i in bad[0].nonzero()} == at


def test_refusals_of_the_binding():
    require_gpu()
    announce("rope refusals")
    z = lambda *s, **k: torch.zeros(*s, device=DEV, **k)  # noqa: E731
    x, q, k, v = z(2, 3, 4 * 64), z(2, 3, 2, 64), z(2, 3, 1, 64), z(2, 3, 1, 64)
    f, p = freqs(64).to(DEV), z(2, dtype=torch.int32)
    for kw in (dict(x=x[:, :2]), dict(q=q[:, :, :1].contiguous()), dict(freq=f.float()),
               dict(freq=f.cpu()), dict(pos=p.long()), dict(pos=p[:1]), dict(v=v.bfloat16()),
               dict(lens=p.long()), dict(q=None), dict(k=z(2, 3, 64)), dict(v=None),
               dict(freq=f[None])):
        with pytest.raises((ValueError, TypeError)):
            gdr.gdr_rope(**{**dict(x=x, freq=f, pos=p, q=q, k=k, v=v), **kw})
    with pytest.raises(gdr.GdrError):
        gdr.gdr_rope(x, freqs(66).to(DEV), p, q, k, v)
    with pytest.raises(gdr.GdrError):
        gdr.gdr_rope(x, f, p, q, v, v)
    gdr.gdr_rope(x[:, :0], f, p, q[:, :0], k[:, :0], v[:, :0])
