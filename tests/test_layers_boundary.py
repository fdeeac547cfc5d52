"""The C ABI of the convolution, the scan and the 8-bit cache without a GPU: bad
arguments are refused with the documented status before anything is launched,
and the binding refuses tensors that do not fit the call."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from gated_delta_rule_40_amd.binding import gdr_conv_dims, gdr_kv_dims, gdr_ssm_dims

E = dict(OK=0, NULL=-1, SHAPE=-2, DTYPE=-3, UNSUPPORTED=-4, WORKSPACE=-5, ALIAS=-7, ALIGN=-8)
M = 0x1000000
A = [M * (i + 1) for i in range(24)]  # fake, aligned, far apart: never dereferenced


def conv(step=False, B=2, T=5, W=4, c=(64, 32, 16), io=1, act=1, x=A[0], stride=None, w=A[1],
         bias=A[2], lens=None, s_in=A[3], s_out=A[4], y=(A[5], A[6], A[7]), dims=True):
    lib = gdr.load_library()
    d = gdr_conv_dims(B, T, W, *c) if dims else None
    stride = sum(c) if stride is None else stride
    if step:
        return lib.gdr_conv_step(d, io, act, x, stride, w, bias, s_out, y[0], None)
    return lib.gdr_conv_prefill(d, io, act, x, stride, w, bias, lens, s_in, s_out, *y, None)


# Every case fails validation or has nothing to launch: the addresses are fake.
@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("case,expect", [
    (dict(dims=False), "NULL"), (dict(io=2), "DTYPE"), (dict(act=2), "DTYPE"),
    (dict(B=-1), "SHAPE"), (dict(c=(0, 8, 8)), "SHAPE"), (dict(c=(8, 0, 8)), "SHAPE"),
    (dict(c=(8, -8, 8), stride=8), "SHAPE"), (dict(stride=111), "SHAPE"),
    (dict(c=(2 ** 31 - 1, 8, 8), stride=2 ** 32), "SHAPE"),
    (dict(B=2 ** 31 - 1, c=(2 ** 20, 0, 0)), "SHAPE"),
    (dict(stride=2 ** 62), "SHAPE"),
    (dict(W=1), "UNSUPPORTED"), (dict(W=5), "UNSUPPORTED"),
    (dict(x=None), "NULL"), (dict(w=None), "NULL"), (dict(s_out=None), "NULL"),
    (dict(y=(None, A[6], A[7])), "NULL"),
    (dict(x=A[0] + 1), "ALIGN"), (dict(w=A[1] + 4), "ALIGN"), (dict(s_out=A[4] + 8), "ALIGN"),
    (dict(y=(A[5] + 2, A[6], A[7])), "ALIGN"), (dict(bias=A[2] + 2), "ALIGN"),
    (dict(y=(A[0], A[6], A[7])), "ALIAS"), (dict(y=(A[4], A[6], A[7])), "ALIAS"),
    (dict(s_out=A[0]), "ALIAS"), (dict(s_out=A[1]), "ALIAS"), (dict(s_out=A[2]), "ALIAS"),
    (dict(B=0), "OK"),
])
def test_conv_refusals(step, case, expect):
    assert conv(step, **case) == E[expect]


@pytest.mark.parametrize("case,expect", [
    (dict(T=-1), "SHAPE"), (dict(T=2 ** 31 - 1, B=2 ** 31 - 1), "SHAPE"),
    (dict(T=2 ** 31 - 8, B=1, c=(4, 0, 0)), "SHAPE"),               # the last tile's end
    (dict(y=(A[5], None, A[7])), "NULL"), (dict(y=(A[5], A[6], None)), "NULL"),
    (dict(y=(A[5], A[5], A[7])), "ALIAS"), (dict(y=(A[5], A[6], A[6] + 16)), "ALIAS"),
    (dict(s_out=A[3] + 16), "ALIAS"), (dict(y=(A[3], A[6], A[7])), "ALIAS"),
    (dict(lens=A[5]), "ALIAS"), (dict(lens=A[8] + 2), "ALIGN"),
    (dict(stride=200, y=(A[0] + 16 * 120, A[6], A[7])), "ALIAS"),   # between strided rows
    (dict(T=0, s_in=A[4]), "OK"),
])
def test_conv_prefill_refusals(case, expect):
    assert conv(False, **case) == E[expect]


def ssm(step=False, B=2, T=70, G=2, H=4, N=32, P=64, io=1, x=A[0], b=A[1], c=A[2], dt=A[3],
        Al=A[4], db=A[5], D=A[6], lens=None, s_in=A[8], s_out=A[9], y=A[10], ws=A[12],
        ws_bytes=None, dims=True):
    lib = gdr.load_library()
    d = gdr_ssm_dims(B, T, G, H, N, P) if dims else None
    if step:
        return lib.gdr_ssm_step(d, io, x, dt, Al, db, D, s_out, y, None)
    if ws_bytes is None:
        ws_bytes = lib.gdr_ssm_workspace_size(d, io)
    return lib.gdr_ssm_prefill(d, io, x, b, c, dt, Al, db, D, lens, s_in, s_out, y, ws, ws_bytes,
                               None)


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("case,expect", [
    (dict(dims=False), "NULL"), (dict(io=7), "DTYPE"), (dict(B=-1), "SHAPE"), (dict(G=0), "SHAPE"),
    (dict(G=3), "SHAPE"), (dict(N=0), "SHAPE"), (dict(N=48), "UNSUPPORTED"),
    (dict(P=8), "UNSUPPORTED"), (dict(P=256), "UNSUPPORTED"),
    (dict(B=2 ** 20, H=2 ** 10), "SHAPE"),
    (dict(B=1, H=2 ** 17, P=128), "SHAPE"),     # a chunk's rows past 32-bit offsets
    (dict(B=1, G=2 ** 20, H=2 ** 20, N=128, P=16), "SHAPE"),
    (dict(x=None), "NULL"), (dict(dt=None), "NULL"), (dict(Al=None), "NULL"),
    (dict(s_out=None), "NULL"), (dict(y=None), "NULL"),
    (dict(x=A[0] + 8), "ALIGN"), (dict(y=A[10] + 4), "ALIGN"), (dict(s_out=A[9] + 8), "ALIGN"),
    (dict(dt=A[3] + 2), "ALIGN"), (dict(D=A[6] + 1), "ALIGN"),
    (dict(y=A[0]), "ALIAS"), (dict(y=A[9]), "ALIAS"), (dict(s_out=A[0]), "ALIAS"),
    (dict(s_out=A[3]), "ALIAS"), (dict(y=A[4]), "ALIAS"), (dict(y=A[5]), "ALIAS"),
    (dict(y=A[6]), "ALIAS"),
    (dict(B=0), "OK"),
])
def test_ssm_refusals(step, case, expect):
    assert ssm(step, **case) == E[expect]


@pytest.mark.parametrize("case,expect", [
    (dict(T=-1), "SHAPE"), (dict(T=2 ** 31 - 1, H=2 ** 12), "SHAPE"),
    (dict(b=None), "NULL"), (dict(c=None), "NULL"), (dict(b=A[1] + 8), "ALIGN"),
    (dict(lens=A[7] + 1), "ALIGN"), (dict(s_in=A[8] + 4), "ALIGN"),
    (dict(y=A[1]), "ALIAS"), (dict(y=A[2]), "ALIAS"), (dict(y=A[8]), "ALIAS"),
    (dict(s_out=A[8] + 64), "ALIAS"), (dict(lens=A[10]), "ALIAS"), (dict(lens=A[9]), "ALIAS"),
    (dict(T=0, s_in=A[9]), "OK"),
])
def test_ssm_prefill_refusals(case, expect):
    assert ssm(False, **case) == E[expect]


def kv(attn=False, B=2, T=3, Hq=8, Hkv=2, D=64, page=32, n_pages=40, per=9, io=1, k=A[0], v=A[1],
       table=A[2], pos=A[3], lens=None, kc=A[5], vc=A[6], ks=A[7], vs=A[8], o=A[9], ws=A[12],
       ws_bytes=None, dims=True):
    lib = gdr.load_library()
    d = gdr_kv_dims(B, T, Hq, Hkv, D, page, n_pages, per) if dims else None
    if not attn:
        return lib.gdr_kv_append(d, io, k, v, table, pos, lens, kc, vc, ks, vs, None)
    if ws_bytes is None:
        ws_bytes = lib.gdr_attn_workspace_size(d, io) if dims else 0
    return lib.gdr_attn_cached(d, io, k, kc, vc, ks, vs, table, pos, lens, o, 0.1, ws, ws_bytes,
                               None)


@pytest.mark.parametrize("attn", [False, True])
@pytest.mark.parametrize("case,expect", [
    (dict(dims=False), "NULL"), (dict(io=-1), "DTYPE"), (dict(B=-1), "SHAPE"), (dict(T=-2), "SHAPE"),
    (dict(Hkv=0), "SHAPE"), (dict(per=-1), "SHAPE"), (dict(n_pages=-1), "SHAPE"),
    (dict(D=96), "UNSUPPORTED"), (dict(D=256), "UNSUPPORTED"), (dict(page=48), "UNSUPPORTED"),
    (dict(page=256), "UNSUPPORTED"), (dict(page=8), "UNSUPPORTED"),
    (dict(B=2 ** 22), "SHAPE"), (dict(per=2 ** 26 + 1), "SHAPE"),
    (dict(per=2 ** 26 - 1), "SHAPE"),              # the last step's end past 32 bits
    (dict(k=None), "NULL"), (dict(table=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(kc=None), "NULL"), (dict(vc=None), "NULL"), (dict(ks=None), "NULL"),
    (dict(vs=None), "NULL"),
    (dict(k=A[0] + 8), "ALIGN"), (dict(kc=A[5] + 8), "ALIGN"), (dict(vc=A[6] + 1), "ALIGN"),
    (dict(ks=A[7] + 2), "ALIGN"), (dict(table=A[2] + 2), "ALIGN"), (dict(pos=A[3] + 1), "ALIGN"),
    (dict(lens=A[4] + 3), "ALIGN"),
    (dict(B=0), "OK"), (dict(T=0), "OK"),
])
def test_kv_refusals(attn, case, expect):
    assert kv(attn, **case) == E[expect]


@pytest.mark.parametrize("attn,case,expect", [
    (False, dict(v=None), "NULL"), (False, dict(v=A[1] + 2), "ALIGN"),
    (False, dict(kc=A[0]), "ALIAS"), (False, dict(vc=A[5]), "ALIAS"),
    (False, dict(ks=A[8]), "ALIAS"), (False, dict(vs=A[5]), "ALIAS"),
    (False, dict(pos=A[7]), "ALIAS"), (False, dict(table=A[6]), "ALIAS"),
    (False, dict(n_pages=0), "OK"), (False, dict(per=0), "OK"),
    (True, dict(Hq=7), "SHAPE"), (True, dict(Hq=0), "SHAPE"), (True, dict(o=None), "NULL"),
    (True, dict(o=A[9] + 4), "ALIGN"), (True, dict(o=A[0]), "ALIAS"), (True, dict(o=A[5]), "ALIAS"),
    (True, dict(o=A[6]), "ALIAS"), (True, dict(o=A[2]), "ALIAS"), (True, dict(o=A[3]), "ALIAS"),
    (True, dict(o=A[7]), "ALIAS"), (True, dict(lens=A[9]), "ALIAS"),
])
def test_kv_refusals_of_one_entry_point(attn, case, expect):
    assert kv(attn, **case) == E[expect]


def test_size_queries_give_zero_for_refused_sizes():
    for d in ((2, -1, 1, 2, 16, 16), (2, 5, 3, 4, 16, 16), (2, 5, 1, 2, 24, 16)):
        assert gdr.gdr_ssm_workspace_size(*d, torch.bfloat16) == 0
    assert gdr.gdr_attn_workspace_size(2, 1, 7, 2, 64, 16, 4, torch.bfloat16) == 0
    assert gdr.gdr_attn_workspace_size(2, 1, 8, 2, 80, 16, 4, torch.bfloat16) == 0
    with pytest.raises(ValueError):
        gdr.gdr_ssm_workspace_size(1, 1, 1, 1, 16, 16, torch.float16)


def test_binding_refuses_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="expected a GPU"):
        gdr.gdr_conv_step(z(2, 8), z(8, 4), None, z(2, 3, 8), z(2, 8))
    with pytest.raises(ValueError, match="expected a GPU"):
        gdr.gdr_ssm_step(z(2, 96), z(2, 2), z(2), None, None, z(2, 2, 16, 16), z(2, 2, 16),
                         G=1, H=2, N=16, P=16)
    with pytest.raises(ValueError, match="dimensions"):
        gdr.gdr_kv_append(z(2, 2, 64), z(2, 2, 64), None, None, None, None, None, None)
    with pytest.raises(TypeError):
        gdr.gdr_conv_step(None, None, None, None, None)


def test_binding_checks_every_property_of_a_tensor():
    from gated_delta_rule_40_amd.binding import _opt, _ptr
    t = torch.zeros(3, 4)
    cpu, f32 = torch.device("cpu"), torch.float32
    assert _ptr(t, "t", (3, 4), f32, cpu) == t.data_ptr()
    assert _ptr(torch.nn.Parameter(t), "t", t.shape, f32, cpu) == t.data_ptr()
    assert _opt(None, "t", (3, 4), f32, cpu) is None
    assert _opt(t, "t", (3, 4), f32, cpu) == t.data_ptr()
    for args, error, text in [
            ((t, "t", (4, 3), f32, cpu), ValueError, "shape"),
            ((t, "t", (12,), f32, cpu), ValueError, "shape"),
            ((t, "t", (3, 2 ** 70), f32, cpu), ValueError, "shape"),
            ((t, "t", (3, 4), torch.bfloat16, cpu), ValueError, "dtype"),
            ((t, "t", (3, 4), f32, torch.device("cuda", 0)), ValueError, "is on cpu"),
            ((t.t(), "t", (4, 3), f32, cpu), ValueError, "contiguous"),
            ((t.to_sparse(), "t", (3, 4), f32, cpu), (ValueError, RuntimeError), None),
            ((None, "t", (3, 4), f32, cpu), TypeError, "torch.Tensor"),
            ((5, "t", (3, 4), f32, cpu), TypeError, "torch.Tensor")]:
        with pytest.raises(error, match=text):
            _ptr(*args)
    with pytest.raises(TypeError):
        _ptr(t)


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 70, -2 ** 31 - 1])
def test_binding_refuses_sizes_past_32_bits(big):
    """Passed on as they are they would wrap: 2^32 + 70 tokens would be 70."""
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="T = .* does not fit 32 bits"):
        gdr.gdr_ssm_workspace_size(1, big, 1, 8, 128, 64, bf)
    with pytest.raises(ValueError, match="max_pages = .* does not fit 32 bits"):
        gdr.gdr_attn_workspace_size(1, 1, 8, 2, 128, 16, big, bf)
    with pytest.raises(ValueError, match="T = .* does not fit 32 bits"):
        gdr.gdr_prefill_workspace_size(1, big, 1, 2, 64, 64, 32, bf, gdr.GDR_GATE_SCALAR)
