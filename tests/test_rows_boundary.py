"""The C ABI of the norms, the 8-bit product and the rotary positions without a GPU:
bad arguments are refused with the documented status before anything is launched, the
binding refuses tensors that do not fit the call, and the frequencies are those of
their formulas."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from gated_delta_rule_40_amd.binding import (gdr_matmul_dims, gdr_norm_dims, gdr_rope_dims,
                                             gdr_rope_scaling)

E = dict(OK=0, NULL=-1, SHAPE=-2, DTYPE=-3, UNSUPPORTED=-4, WORKSPACE=-5, ALIAS=-7, ALIGN=-8)
M = 0x1000000
A = [M * (i + 1) for i in range(24)]  # fake, aligned, far apart: never dereferenced


def norm(R=3, H=2, D=128, io=1, x=A[0], stride=None, res=1, residual=None, order=0, gate=A[1],
         gstride=None, weight=A[2], eps=1e-6, y=A[3], codes=A[4], scales=A[5], dims=True):
    lib = gdr.load_library()
    d = gdr_norm_dims(R, H, D) if dims else None
    stride = H * D if stride is None else stride
    gstride = H * D if gstride is None else gstride
    return lib.gdr_rms_norm(d, io, x, stride, res, residual, order, gate, gstride, weight, eps, y,
                            codes, scales, None)


# Every case fails validation or has nothing to launch: the addresses are fake.
@pytest.mark.parametrize("case,expect", [
    (dict(dims=False), "NULL"), (dict(io=2), "DTYPE"), (dict(order=3), "DTYPE"),
    (dict(order=-1), "DTYPE"), (dict(res=2, residual=A[6]), "DTYPE"),
    (dict(R=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(D=0), "SHAPE"), (dict(D=-128), "SHAPE"),
    (dict(H=2 ** 24, D=128), "SHAPE"), (dict(stride=255), "SHAPE"), (dict(stride=-256), "SHAPE"),
    (dict(R=2 ** 27), "SHAPE"), (dict(R=2 ** 24, H=1, D=4096), "SHAPE"),
    (dict(R=2 ** 22, H=4, D=384), "SHAPE"), (dict(H=2 ** 24 - 1, D=128), "SHAPE"),
    (dict(R=2 ** 20, stride=2 ** 50), "SHAPE"),
    (dict(order=1, gstride=255), "SHAPE"), (dict(order=2, R=2 ** 20, gstride=2 ** 50), "SHAPE"),
    (dict(H=1, D=32769), "UNSUPPORTED"), (dict(D=48), "UNSUPPORTED"), (dict(D=8), "UNSUPPORTED"),
    (dict(D=200), "UNSUPPORTED"),
    (dict(eps=0.0), "UNSUPPORTED"), (dict(eps=-1e-6), "UNSUPPORTED"),
    (dict(eps=math.nan), "UNSUPPORTED"), (dict(eps=math.inf), "UNSUPPORTED"),
    (dict(order=1, residual=A[6]), "UNSUPPORTED"), (dict(order=2, residual=A[6]), "UNSUPPORTED"),
    (dict(x=None), "NULL"), (dict(order=1, gate=None), "NULL"), (dict(codes=None), "NULL"),
    (dict(scales=None), "NULL"), (dict(y=None, codes=None, scales=None), "NULL"),
    (dict(x=A[0] + 1), "ALIGN"), (dict(io=0, x=A[0] + 2), "ALIGN"), (dict(y=A[3] + 8), "ALIGN"),
    (dict(order=1, gate=A[1] + 1), "ALIGN"), (dict(weight=A[2] + 2), "ALIGN"),
    (dict(codes=A[4] + 8), "ALIGN"), (dict(scales=A[5] + 2), "ALIGN"),
    (dict(residual=A[6] + 4), "ALIGN"),
    (dict(y=A[0]), "ALIAS"), (dict(codes=A[0] + 16), "ALIAS"), (dict(scales=A[2]), "ALIAS"),
    (dict(y=A[4]), "ALIAS"), (dict(residual=A[0]), "ALIAS"), (dict(residual=A[3]), "ALIAS"),
    (dict(scales=A[4] + 32), "ALIAS"), (dict(order=1, y=A[1]), "ALIAS"),
    (dict(stride=1000, y=A[0] + 1024), "ALIAS"),          # between strided rows
    (dict(R=0), "OK"), (dict(R=0, x=None, y=None, codes=None), "OK"),
])
def test_norm_refusals(case, expect):
    assert norm(**case) == E[expect]


def quant(R=3, H=2, D=128, io=1, x=A[0], stride=None, codes=A[4], scales=A[5], dims=True):
    lib = gdr.load_library()
    d = gdr_norm_dims(R, H, D) if dims else None
    return lib.gdr_quant_rows(d, io, x, H * D if stride is None else stride, codes, scales, None)


@pytest.mark.parametrize("case,expect", [
    (dict(dims=False), "NULL"), (dict(io=2), "DTYPE"), (dict(R=-1), "SHAPE"),
    (dict(stride=255), "SHAPE"), (dict(D=48), "UNSUPPORTED"), (dict(x=None), "NULL"),
    (dict(codes=None), "NULL"), (dict(scales=None), "NULL"), (dict(x=A[0] + 1), "ALIGN"),
    (dict(codes=A[4] + 4), "ALIGN"), (dict(scales=A[5] + 1), "ALIGN"), (dict(codes=A[0]), "ALIAS"),
    (dict(scales=A[4]), "ALIAS"), (dict(R=0), "OK"),
])
def test_quant_refusals(case, expect):
    assert quant(**case) == E[expect]


def matmul(m=5, n=300, k=272, io=1, x=A[0], sx=A[1], w=A[2], sw=A[3], bias=A[4], y=A[5],
           dims=True):
    lib = gdr.load_library()
    return lib.gdr_matmul_fp8(gdr_matmul_dims(m, n, k) if dims else None, io, x, sx, w, sw, bias,
                              y, None)


@pytest.mark.parametrize("case,expect", [
    (dict(dims=False), "NULL"), (dict(io=3), "DTYPE"), (dict(m=-1), "SHAPE"), (dict(n=-1), "SHAPE"),
    (dict(k=-16), "SHAPE"), (dict(m=2 ** 30, n=2 ** 20), "SHAPE"),
    (dict(m=2 ** 31 - 1, n=1), "SHAPE"), (dict(m=1, n=2 ** 31 - 1), "SHAPE"),
    (dict(k=264), "UNSUPPORTED"), (dict(k=2 ** 20 + 16), "UNSUPPORTED"),
    (dict(x=None), "NULL"), (dict(sx=None), "NULL"), (dict(w=None), "NULL"),
    (dict(sw=None), "NULL"), (dict(y=None), "NULL"), (dict(k=0, y=None), "NULL"),
    (dict(x=A[0] + 8), "ALIGN"), (dict(w=A[2] + 4), "ALIGN"), (dict(y=A[5] + 8), "ALIGN"),
    (dict(sx=A[1] + 2), "ALIGN"), (dict(sw=A[3] + 1), "ALIGN"), (dict(bias=A[4] + 2), "ALIGN"),
    (dict(y=A[0]), "ALIAS"), (dict(y=A[1]), "ALIAS"), (dict(y=A[2]), "ALIAS"),
    (dict(y=A[3]), "ALIAS"), (dict(y=A[4]), "ALIAS"),
    (dict(m=0), "OK"), (dict(n=0), "OK"),
])
def test_matmul_refusals(case, expect):
    assert matmul(**case) == E[expect]


@pytest.mark.parametrize("call,case", [
    (norm, dict(R=2 ** 22, H=1, D=16384, stride=16384)),  # 1024 threads a row
    (norm, dict(R=2 ** 22, H=1, D=16384, stride=16384, codes=None, scales=None)),
    (quant, dict(R=2 ** 20, H=4, D=8320)),
    (matmul, dict(m=1, n=2 ** 27, k=16)),                 # 512 threads for 16 outputs
    (matmul, dict(m=16, n=2 ** 27, k=16, io=0)),
])
def test_launches_of_2_32_threads_are_refused(call, case):
    assert call(**case) == E["SHAPE"]


def rope(B=2, T=5, Hq=4, Hkv=2, D=64, R=64, io=1, pairs=0, x=A[0], stride=None, freq=A[1],
         pos=A[2], lens=None, q=A[3], k=A[4], v=A[5], dims=True):
    lib = gdr.load_library()
    d = gdr_rope_dims(B, T, Hq, Hkv, D, R) if dims else None
    stride = (Hq + 2 * Hkv) * D if stride is None else stride
    return lib.gdr_rope(d, io, pairs, x, stride, freq, 1.0, pos, lens, q, k, v, None)


@pytest.mark.parametrize("case,expect", [
    (dict(dims=False), "NULL"), (dict(io=2), "DTYPE"), (dict(pairs=2), "DTYPE"),
    (dict(B=-1), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(Hq=0), "SHAPE"), (dict(Hkv=0), "SHAPE"),
    (dict(R=66), "SHAPE"), (dict(R=-2), "SHAPE"), (dict(R=31), "SHAPE"), (dict(D=0, R=0), "SHAPE"),
    (dict(stride=8 * 64 - 1), "SHAPE"), (dict(stride=2 ** 60), "SHAPE"),
    (dict(B=2 ** 12, T=2 ** 12), "SHAPE"), (dict(Hq=2 ** 26), "SHAPE"),
    (dict(D=60, R=32), "UNSUPPORTED"), (dict(D=520), "UNSUPPORTED"),
    (dict(x=None), "NULL"), (dict(pos=None), "NULL"), (dict(q=None), "NULL"),
    (dict(k=None), "NULL"), (dict(freq=None), "NULL"),
    (dict(x=A[0] + 1), "ALIGN"), (dict(freq=A[1] + 4), "ALIGN"), (dict(pos=A[2] + 2), "ALIGN"),
    (dict(lens=A[6] + 1), "ALIGN"), (dict(q=A[3] + 8), "ALIGN"), (dict(k=A[4] + 8), "ALIGN"),
    (dict(v=A[5] + 8), "ALIGN"),
    (dict(q=A[0]), "ALIAS"), (dict(k=A[3]), "ALIAS"), (dict(v=A[4]), "ALIAS"),
    (dict(q=A[1]), "ALIAS"), (dict(v=A[2]), "ALIAS"), (dict(lens=A[5]), "ALIAS"),
    (dict(B=0), "OK"), (dict(T=0), "OK"), (dict(v=None, stride=6 * 64 - 1), "SHAPE"),
])
def test_rope_refusals(case, expect):
    assert rope(**case) == E[expect]


# ---- frequencies ------------------------------------------------------------
def freqs(R=128, base=10000.0, **kw):
    return gdr.gdr_rope_freqs(R, base, **kw)


@pytest.mark.parametrize("R", [2, 6, 64, 128, 512])
def test_frequencies_without_scaling(R):
    f, m = freqs(R, 500000.0)
    assert m == 1.0 and f.dtype == torch.float64
    for i in range(R // 2):
        assert math.isclose(f[i].item(), 500000.0 ** (-2 * i / R), rel_tol=1e-14)


def test_frequencies_stretched_evenly():
    f, _ = freqs()
    g, m = freqs(kind=gdr.GDR_ROPE_LINEAR, factor=4.0)
    assert m == 1.0 and torch.allclose(g, f / 4, rtol=1e-14, atol=0)


@pytest.mark.parametrize("R,factor", [(128, 8.0), (64, 2.5), (4, 16.0)])
def test_frequencies_of_a_larger_base(R, factor):
    """The first frequency stays, the last is divided by the factor."""
    f, _ = freqs(R)
    g, m = freqs(R, kind=gdr.GDR_ROPE_BASE, factor=factor)
    assert m == 1.0 and g[0] == 1.0
    assert math.isclose(g[-1].item(), f[-1].item() / factor, rel_tol=1e-13)


def test_frequencies_by_turns():
    ctx, low, high, k = 8192.0, 1.0, 4.0, 8.0
    f, _ = freqs(base=500000.0)
    g, m = freqs(base=500000.0, kind=gdr.GDR_ROPE_TURNS, factor=k, context=ctx, low=low, high=high)
    assert m == 1.0
    seen = set()
    for a, b in zip(f.tolist(), g.tolist()):
        turns = ctx * a / (2 * math.pi)
        if turns < low:
            want, part = a / k, "far"
        elif turns > high:
            want, part = a, "near"
        else:
            u = (turns - low) / (high - low)
            want, part = (1 - u) * a / k + u * a, "between"
        seen.add(part)
        assert math.isclose(b, want, rel_tol=1e-13)
    assert seen == {"far", "near", "between"}


def test_frequencies_by_index():
    R, base, k, ctx, low, high = 128, 10000.0, 16.0, 4096.0, 1.0, 32.0
    f, _ = freqs(R, base)
    g, m = freqs(R, base, kind=gdr.GDR_ROPE_INDEX, factor=k, context=ctx, low=low, high=high)
    assert math.isclose(m, 0.1 * math.log(k) + 1, rel_tol=1e-6)

    def index(turns):
        return R * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(base))

    first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), R - 1)
    assert 0 < first < last < R // 2
    for i, (a, b) in enumerate(zip(f.tolist(), g.tolist())):
        stretched = min(max((i - first) / (last - first), 0), 1)
        assert math.isclose(b, a / k * stretched + a * (1 - stretched), rel_tol=1e-13)


def test_frequencies_by_index_of_a_short_context():
    """Where both ends fall on index 0 the ramp is a step: only index 0 stays."""
    f, _ = freqs(8)
    g, _ = freqs(8, kind=gdr.GDR_ROPE_INDEX, factor=2.0, context=1.0, low=1.0, high=32.0)
    assert g[0] == 1.0 and torch.allclose(g[1:], f[1:] / 2, rtol=1e-14, atol=0)


@pytest.mark.parametrize("kw,status", [
    (dict(R=3), "SHAPE"), (dict(base=1.0), "UNSUPPORTED"), (dict(base=math.inf), "UNSUPPORTED"),
    (dict(base=math.nan), "UNSUPPORTED"), (dict(kind=5), "DTYPE"), (dict(kind=-1), "DTYPE"),
    (dict(kind=1, factor=0.5), "UNSUPPORTED"), (dict(kind=1, factor=math.inf), "UNSUPPORTED"),
    (dict(kind=2, R=2, factor=2.0), "UNSUPPORTED"),
    (dict(kind=3, factor=2.0, context=0.0), "UNSUPPORTED"),
    (dict(kind=3, factor=2.0, context=10.0, low=4.0, high=4.0), "UNSUPPORTED"),
    (dict(kind=4, factor=2.0, context=10.0, low=0.0), "UNSUPPORTED"),
])
def test_frequency_refusals(kw, status):
    with pytest.raises(gdr.GdrError) as e:
        freqs(**kw)
    assert e.value.status == E[status]


def test_frequency_refusals_of_the_c_abi():
    lib = gdr.load_library()
    out = (ctypes.c_double * 256)()
    addr = ctypes.addressof(out)
    assert lib.gdr_rope_freqs(64, 1e4, None, None, None) == E["NULL"]
    assert lib.gdr_rope_freqs(514, 1e4, None, addr, None) == E["SHAPE"]
    assert lib.gdr_rope_freqs(0, 1e4, None, addr, None) == E["SHAPE"]
    assert lib.gdr_rope_freqs(64, 1e4, None, addr, None) == 0 and out[0] == 1.0 and out[32] == 0.0
    s = gdr_rope_scaling(0, math.nan, 0, 0, 0)          # factor is not looked at
    assert lib.gdr_rope_freqs(64, 1e4, ctypes.byref(s), addr, None) == 0
    for R in (0, 514, -2):
        with pytest.raises(ValueError):
            freqs(R)


def test_binding_refuses_what_does_not_fit():
    z, f8 = torch.zeros, torch.float8_e4m3fn
    x, c = z(2, 128), z(2, 128, dtype=f8)
    with pytest.raises(ValueError, match="expected a GPU"):
        gdr.gdr_rms_norm(x, z(128), z(2, 128))
    with pytest.raises(ValueError, match="expected a GPU"):
        gdr.gdr_quant_rows(x, c, z(2, 1))
    with pytest.raises(ValueError, match="expected a GPU"):
        gdr.gdr_matmul_fp8(c, z(2, 1), c, z(1, 1), z(2, 2))
    with pytest.raises(ValueError, match="expected a GPU"):
        gdr.gdr_rope(z(1, 2, 192), z(32, dtype=torch.float64), z(1), z(1, 2, 1, 64),
                     z(1, 2, 1, 64), z(1, 2, 1, 64))
    with pytest.raises(ValueError, match="dimensions"):
        gdr.gdr_rms_norm(z(2, 3, 4))
    with pytest.raises(TypeError):
        gdr.gdr_quant_rows(None, c, z(2, 1))
    with pytest.raises(TypeError):
        gdr.gdr_matmul_fp8(c, z(2, 1), c, z(1, 1), None)
