"""The short causal convolution on the GPU against its 64-bit form."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu


def inputs(seed, B, T, C, W, io):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return (r(B, T, C).to(io_dtype(io)), r(C, W) * 0.6, r(C) * 0.3, r(B, W - 1, C).to(io_dtype(io)))


def up(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


# (B, T, widths): one token, fewer tokens than taps, around the tile of a
# thread (16), odd widths (one channel a thread), one to three outputs.
SHAPES = [(1, 1, (8,)), (2, 2, (16, 8)), (3, 3, (8, 8, 8)), (1, 15, (64,)), (2, 16, (24, 40)),
          (1, 17, (8, 16, 264)), (2, 33, (7, 5, 3)), (3, 50, (1,)), (1, 130, (100, 28)),
          (2, 65, (512, 256, 1024)), (1, 300, (37, 91))]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,widths", SHAPES)
def test_prefill(B, T, widths, W, io):
    require_gpu()
    announce(f"conv prefill B={B} T={T} widths={widths} W={W} io={io}")
    C = sum(widths)
    x, w, bias, s0 = inputs(B * 1000 + T, B, T, C, W, io)
    for silu, use_bias, use_state, lens in [(True, True, True, None), (False, False, False, None),
                                            (True, False, True, [T, 0, T // 2][:B]),
                                            (True, True, False, [1, T + 5, -3][:B])]:
        bb, ss = (bias if use_bias else None), (s0 if use_state else None)
        want, mag, st = ref.conv(x, w, bb, ss, silu, lens)
        gx, gw, gb, gs = up(x, w, bb, ss)
        outs = [torch.full((B, T, c), 7.0, dtype=x.dtype, device=DEV) for c in widths]
        s_out = torch.full((B, W - 1, C), 7.0, dtype=x.dtype, device=DEV)
        gl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
        gdr.gdr_conv_prefill(gx, gw, gb, gs, s_out, outs, silu=silu, lens=gl)
        got = torch.cat([o.cpu() for o in outs], -1)
        bound = ref.conv_bound(want, mag, x.dtype, W)
        for b, n in enumerate(ref.clip_lens(lens, B, T)):
            assert ref.worst(got[b, :n], want[b, :n], bound[b, :n]) <= 1
            assert (got[b, n:] == 7).all()               # rows behind the end stay as they were
        assert torch.equal(s_out.cpu().to(ref.F64), st)
        if ss is not None:                               # the state in place
            gdr.gdr_conv_prefill(gx, gw, gb, gs, gs, outs, silu=silu, lens=gl)
            assert torch.equal(gs, s_out)
            assert torch.equal(torch.cat([o.cpu() for o in outs], -1), got)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,C", [(1, 8), (1, 1), (5, 96), (3, 77), (64, 1030), (7, 4096)])
def test_steps_equal_prefill(B, C, W, io):
    require_gpu()
    announce(f"conv steps B={B} C={C} W={W} io={io}")
    T = 6
    x, w, bias, s0 = inputs(B * 100 + C, B, T, C, W, io)
    want, mag, st = ref.conv(x, w, bias, s0)
    gx, gw, gb, gs = up(x, w, bias, s0)
    y = torch.empty((B, C), dtype=x.dtype, device=DEV)
    outs, s_out = [torch.empty_like(gx)], torch.empty_like(gs)
    gdr.gdr_conv_prefill(gx, gw, gb, gs, s_out, outs)
    bound = ref.conv_bound(want, mag, x.dtype, W)
    for t in range(T):
        gdr.gdr_conv_step(gx[:, t], gw, gb, gs, y)       # rows T * C apart
        assert ref.worst(y.cpu(), want[:, t], bound[:, t]) <= 1
        assert torch.equal(y, outs[0][:, t])
    assert torch.equal(gs, s_out)
    assert torch.equal(gs.cpu().to(ref.F64), st)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lo,C,width", [(0, 64, 96), (8, 64, 96), (3, 64, 96), (16, 64, 81),
                                        (1, 33, 50)])
def test_slices_of_wider_rows(lo, C, width, io):
    """The input as a slice of a projection's rows: aligned and unaligned starts and strides."""
    require_gpu()
    announce(f"conv slice lo={lo} C={C} width={width} io={io}")
    B, T, W = 2, 21, 4
    rows, w, bias, s0 = inputs(5, B, T, width, W, io)
    w, bias, s0 = w[:C].contiguous(), bias[:C].contiguous(), s0[:, :, :C].contiguous()
    x = rows[:, :, lo: lo + C]
    want, mag, st = ref.conv(x, w, bias, s0)
    g, gw, gb, gs = up(rows, w, bias, s0)
    out = torch.empty((B, T, C), dtype=x.dtype, device=DEV)
    gdr.gdr_conv_prefill(g[:, :, lo: lo + C], gw, gb, gs, gs, [out])
    assert ref.worst(out.cpu(), want, ref.conv_bound(want, mag, x.dtype, W)) <= 1
    assert torch.equal(gs.cpu().to(ref.F64), st)
    # One token a row: the rows lie a whole sequence apart.
    one, st1 = torch.empty((B, 1, C), dtype=x.dtype, device=DEV), up(s0)[0]
    gdr.gdr_conv_prefill(g[:, :1, lo: lo + C], gw, gb, st1, st1, [one])
    assert torch.equal(one, out[:, :1])
    one, st1 = torch.empty((1, 1, C), dtype=x.dtype, device=DEV), up(s0[:1].contiguous())[0]
    gdr.gdr_conv_prefill(g[:1, :1, lo: lo + C], gw, gb, st1, st1, [one])
    assert torch.equal(one, out[:1, :1])
    with pytest.raises(ValueError):
        gdr.gdr_conv_prefill(g[:, :-1, lo: lo + C], gw, gb, gs, gs, [out[:, :-1].contiguous()])
    with pytest.raises(ValueError):
        gdr.gdr_conv_prefill(g[:, :, ::2], gw, gb, gs, gs, [out])


def test_no_tokens_copies_the_state():
    require_gpu()
    announce("conv T=0 and B=0")
    x, w, bias, s0 = inputs(1, 3, 0, 24, 4, "bf16")
    gx, gw, gb, gs = up(x, w, bias, s0)
    out, s_out = torch.empty((3, 0, 24), dtype=x.dtype, device=DEV), torch.full_like(gs, 7)
    gdr.gdr_conv_prefill(gx, gw, gb, gs, s_out, [out])
    assert torch.equal(s_out, gs)
    gdr.gdr_conv_prefill(gx, gw, gb, None, s_out, [out])
    assert (s_out == 0).all()
    gdr.gdr_conv_step(gx[:0, 0] if gx.shape[1] else gx[:0].reshape(0, 24), gw, gb, gs[:0],
                      torch.empty((0, 24), dtype=x.dtype, device=DEV))


def test_what_is_not_finite_stays_in_its_channel():
    require_gpu()
    announce("conv with inf and NaN inputs")
    x, w, bias, s0 = inputs(3, 1, 12, 16, 4, "f32")
    x[0, 4, 3], x[0, 5, 9] = float("nan"), float("inf")
    want, mag, _ = ref.conv(x, w, bias, s0)
    gx, gw, gb, gs = up(x, w, bias, s0)
    out = torch.empty_like(gx)
    gdr.gdr_conv_prefill(gx, gw, gb, gs, gs, [out])
    got = out.cpu()
    fine = torch.ones(16, dtype=torch.bool)
    fine[[3, 9]] = False
    bound = ref.conv_bound(want, mag, x.dtype, 4)
    assert ref.worst(got[:, :, fine], want[:, :, fine], bound[:, :, fine]) <= 1
    assert torch.isnan(got[0, 4:8, 3]).all() and torch.isfinite(got[0, 8:, 3]).all()
    assert not torch.isfinite(got[0, 5:9, 9]).any() or w[9].min() < 0
    assert torch.isfinite(got[0, 9:, 9]).all()


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("io,C", [("f32", 16), ("f32", 15), ("bf16", 16), ("bf16", 13)])
def test_infinite_inputs_follow_the_taps_sign(io, C, silu):
    """An infinite input makes the W tokens of its window infinite with the sign of
    its tap; the sigmoid takes minus infinity to NaN (0 times infinity).  C = 15 and
    13 take one channel a thread."""
    require_gpu()
    announce(f"conv with infinities C={C} io={io} silu={silu}")
    x, w, bias, s0 = inputs(3, 1, 12, C, 4, io)
    w[:, 0], w[:, 1], w[:, 2], w[:, 3] = 0.5, -0.25, 1.5, -2.0
    clean = x.clone()
    x[0, 5, 9], x[0, 2, 4] = math.inf, -math.inf
    want, mag, _ = ref.conv(clean, w, bias, s0, silu=silu)
    bound = ref.conv_bound(want, mag, x.dtype, 4)
    gw, gb, gs = up(w, bias, s0)
    out = torch.empty((1, 12, C), dtype=x.dtype, device=DEV)
    gdr.gdr_conv_prefill(x.to(DEV), gw, gb, gs, gs, [out], silu=silu)
    got = out.cpu().double()
    minus = math.nan if silu else -math.inf
    touched = torch.zeros_like(want, dtype=torch.bool)
    for t, c, plus in ((5, 9, 1), (2, 4, -1)):
        for i in range(4):                                # tap 3 - i meets it i tokens later
            rises = w[c, 3 - i] * plus > 0
            v, e = got[0, t + i, c], math.inf if rises else minus
            assert torch.isnan(v) if math.isnan(e) else v == e, (t + i, c)
            touched[0, t + i, c] = True
    assert ref.worst(got[~touched], want[~touched], bound[~touched]) <= 1
