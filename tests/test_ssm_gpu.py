"""The selective state space scan on the GPU against its 64-bit token recurrence."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def inputs(seed, B, T, G, H, N, P, io, strong=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    dt = io_dtype(io)
    return dict(x=r(B, T, H, P).to(dt), b=r(B, T, G, N).to(dt), c=r(B, T, G, N).to(dt),
                dt=r(B, T, H) * (6.0 if strong else 1.0),
                A_log=torch.log(1 + 15 * torch.rand(H, generator=gen)),
                dt_bias=torch.full((H,), 0.0 if strong else -3.0) + 0.5 * r(H), D=r(H)), \
        0.2 * r(B, H, N, P)


def up(d):
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def prefill(d, s_in, G, lens=None, in_place=False, ws_fill=None):
    """y and the state of one call, every output filled with 7 before it."""
    B, T, H, P = d["x"].shape
    N = d["b"].shape[3]
    g = up(d)
    s = None if s_in is None else s_in.to(DEV)
    s_out = s if in_place else torch.full((B, H, N, P), 7.0, device=DEV)
    y = torch.full_like(g["x"], 7.0)
    size = dict(G=G, H=H, N=N, P=P)
    n = gdr.gdr_ssm_workspace_size(B, T, io_dtype=d["x"].dtype, **size)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None   # NaN as floats
    gl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    gdr.gdr_ssm_prefill(g["x"], g["b"], g["c"], g["dt"], g["A_log"], g["dt_bias"], g["D"], s, s_out,
                        y, ws, lens=gl, **size)
    torch.cuda.synchronize()
    return y.cpu(), s_out.cpu()


def check(d, s_in, got, lens=None):
    B, T = d["x"].shape[:2]
    N, io = d["b"].shape[3], d["x"].dtype
    want, mag, S, M = ref.ssm(**d, state=s_in, lens=lens)
    y, s = got
    # fp32: a term is off by ssm_units at most.  bf16: the output rounds by
    # half a step of its value, and in the chunk form each weight and each
    # state element rounds by half a step of its own before its product.
    bound = ref.ssm_units(T, N) * EPS * mag + 1e-30
    if io == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + mag)
    ns = ref.clip_lens(lens, B, T)
    for b, n in enumerate(ns):
        assert ref.worst(y[b, :n], want[b, :n], bound[b, :n]) <= 1
        assert (y[b, n:] == 7).all()
    assert ref.worst(s, S, ref.ssm_units(T, N) * EPS * M + 1e-30) <= 1
    # Over the whole tensor the roundings add up as independent ones: the
    # output's, the weights' and the state's, each uniform over half a step.
    keep = torch.tensor([[t < n for t in range(T)] for n in ns])
    if keep.any():
        assert ref.rel(y[keep], want[keep]) <= (2.0 ** -8 if io == torch.bfloat16
                                                 else ref.ssm_norm(T, N))
    if S.norm() > 0:
        assert ref.rel(s, S) <= ref.ssm_norm(T, N)


# Around the chunk of 64 tokens, one token, one head, shared and own groups.
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,G,H,N,P", [
    (1, 1, 1, 1, 16, 16), (2, 5, 1, 2, 32, 16), (1, 16, 2, 2, 64, 32), (2, 63, 1, 3, 16, 64),
    (1, 64, 2, 4, 128, 64), (1, 65, 1, 2, 64, 128), (3, 100, 2, 6, 32, 16), (1, 129, 1, 1, 128, 128),
    (2, 200, 4, 4, 16, 32), (1, 321, 1, 5, 128, 32), (2, 257, 1, 2, 32, 128), (1, 640, 1, 8, 64, 64)])
def test_prefill(B, T, G, H, N, P, io):
    require_gpu()
    announce(f"ssm prefill B={B} T={T} G={G} H={H} N={N} P={P} io={io}")
    d, s0 = inputs(T + 7 * N, B, T, G, H, N, P, io)
    check(d, s0, prefill(d, s0, G))
    check(d, None, prefill(d, None, G))
    lens = [T // 2, T + 9, -1][:B]
    check(d, s0, prefill(d, s0, G, lens, in_place=True), lens)
    bare = dict(d, dt_bias=None, D=None)
    check(bare, s0, prefill(bare, s0, G))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("N,P", [(16, 16), (16, 128), (32, 64), (64, 16), (128, 32), (128, 128)])
def test_every_width(N, P, io):
    require_gpu()
    announce(f"ssm widths N={N} P={P} io={io}")
    d, s0 = inputs(N + P, 2, 150, 2, 4, N, P, io)
    check(d, s0, prefill(d, s0, 2, [150, 77]), [150, 77])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_and_mixed_decay(io):
    """Step sizes from about 0 to 20 at rates up to 16: a chunk decays by up to
    e^-1e4 between tokens that hardly decay at all."""
    require_gpu()
    announce(f"ssm strong decay io={io}")
    d, s0 = inputs(5, 2, 200, 1, 4, 32, 32, io, strong=True)
    check(d, s0, prefill(d, s0, 1))
    d["dt"][:, 10:14] = 60.0
    d["dt"][:, 70:74] = -60.0
    check(d, s0, prefill(d, s0, 1))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_weak_decay_keeps_the_first_token(io):
    require_gpu()
    announce(f"ssm weak decay io={io}")
    d, s0 = inputs(6, 1, 700, 1, 2, 16, 32, io)
    d["A_log"] = torch.full((2,), math.log(1e-3))
    d["dt_bias"] = torch.full((2,), -6.0)
    check(d, s0, prefill(d, s0, 1))


@pytest.mark.parametrize("B,H,T", [(1, 2, 4097), (1, 24, 1500), (40, 8, 130)])
def test_few_and_many_workgroups(B, H, T):
    """Long sequences over few heads (cut into parts), and wide batches."""
    require_gpu()
    announce(f"ssm B={B} H={H} T={T}")
    d, s0 = inputs(T, B, T, 1, H, 64, 64, "bf16")
    lens = None if B == 1 else [(i * 37) % (T + 1) for i in range(B)]
    check(d, s0, prefill(d, s0, 1, lens), lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,G,H,N,P", [
    (1, 1, 1, 16, 16), (3, 2, 4, 16, 32), (2, 1, 3, 32, 16), (5, 4, 4, 64, 64), (1, 1, 32, 128, 64),
    (2, 2, 8, 128, 128), (3, 1, 2, 32, 128), (2, 1, 2, 128, 16), (64, 1, 4, 64, 128)])
def test_steps(B, G, H, N, P, io):
    require_gpu()
    announce(f"ssm steps B={B} G={G} H={H} N={N} P={P} io={io}")
    T = 4
    d, s0 = inputs(B + N, B, T, G, H, N, P, io)
    for bare in (False, True):
        d = dict(d, dt_bias=None, D=None) if bare else d
        g, S = up(d), s0.to(DEV)
        y = torch.empty((B, H, P), dtype=g["x"].dtype, device=DEV)
        ys = []
        for t in range(T):
            xbc = torch.cat([g[k][:, t].flatten(1) for k in ("x", "b", "c")], 1).contiguous()
            gdr.gdr_ssm_step(xbc, g["dt"][:, t].contiguous(), g["A_log"], g["dt_bias"], g["D"], S,
                             y, G=G, H=H, N=N, P=P)
            ys.append(y.cpu())
        check(d, s0, (torch.stack(ys, 1), S.cpu()))


def test_step_of_a_large_state():
    """A state of 72 MiB (it passes the caches by): rows against the same rows alone."""
    require_gpu()
    announce("ssm step B=72 H=32 N=128 P=64")
    B, G, H, N, P = 72, 4, 32, 128, 64
    d, s0 = inputs(3, B, 1, G, H, N, P, "bf16")
    g, S = up(d), s0.to(DEV)
    xbc = torch.cat([g[k][:, 0].flatten(1) for k in ("x", "b", "c")], 1).contiguous()
    y = torch.empty((B, H, P), dtype=g["x"].dtype, device=DEV)
    size = dict(G=G, H=H, N=N, P=P)
    dt = g["dt"][:, 0].contiguous()
    for rows in (slice(0, 5), slice(67, 72)):
        part, yp = s0[rows].to(DEV), torch.empty_like(y[rows])
        gdr.gdr_ssm_step(xbc[rows], dt[rows], g["A_log"], g["dt_bias"], g["D"], part, yp, **size)
        whole = S.clone()
        gdr.gdr_ssm_step(xbc, dt, g["A_log"], g["dt_bias"], g["D"], whole, y, **size)
        assert torch.equal(whole[rows], part) and torch.equal(y[rows], yp)
    want, mag, st, M = ref.ssm(**d, state=s0)
    assert ref.worst(y.cpu(), want[:, 0], 2.0 ** -8 * want[:, 0].abs()
                     + ref.ssm_units(1, N) * EPS * mag[:, 0]) <= 1
    assert ref.worst(whole.cpu(), st, ref.ssm_units(1, N) * EPS * M + 1e-30) <= 1


def test_no_tokens_copies_the_state():
    require_gpu()
    announce("ssm T=0 and B=0")
    d, s0 = inputs(2, 2, 0, 1, 2, 32, 32, "bf16")
    _, s = prefill(d, s0, 1)
    assert torch.equal(s, s0)
    _, s = prefill(d, None, 1)
    assert (s == 0).all()
    d, s0 = inputs(2, 0, 5, 1, 2, 32, 32, "bf16")
    prefill(d, s0, 1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_nan_behind_a_rows_end_does_not_matter(io):
    require_gpu()
    announce(f"ssm NaN padding io={io}")
    d, s0 = inputs(9, 2, 150, 1, 2, 32, 32, io)
    lens = [70, 129]
    clean = prefill(d, s0, 1, lens)
    for k in ("x", "b", "c", "dt"):
        for i, n in enumerate(lens):
            d[k][i, n:] = float("nan")
    got = prefill(d, s0, 1, lens)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 200])
def test_nan_token_does_not_reach_earlier_ones(T, io):
    require_gpu()
    announce(f"ssm NaN token T={T} io={io}")
    d, s0 = inputs(10, 1, T, 2, 4, 32, 64, io)
    clean, _ = prefill(d, s0, 2)
    at = T // 2 + 3
    d["x"][0, at, 1, 5] = float("nan")       # head 1, column 5
    y, s = prefill(d, s0, 2)
    assert torch.equal(y[:, :at], clean[:, :at])
    assert torch.equal(y[:, :, [0, 2, 3]], clean[:, :, [0, 2, 3]])
    assert torch.isnan(y[0, at:, 1, 5]).all() and torch.isnan(s[0, 1, :, 5]).all()
    cols = [p for p in range(64) if p != 5]
    assert torch.equal(y[..., cols], clean[..., cols])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 8, 200])
def test_dt_of_minus_infinity_leaves_the_state(T, io):
    """softplus(-inf) = 0: such a token neither decays nor writes, and y = S^T C + D x."""
    require_gpu()
    announce(f"ssm dt = -inf T={T} io={io}")
    d, s0 = inputs(11, 2, T, 1, 2, 32, 32, io)
    d["dt"][0, T // 2:] = -math.inf
    d["dt"][1, ::3] = -math.inf
    check(d, s0, prefill(d, s0, 1))


@pytest.mark.parametrize("B,G,H,N,P,T,lens,io", [
    (1, 1, 128, 128, 64, 449, None, "f32"), (1, 1, 128, 128, 64, 449, [40], "f32"),
    (1, 1, 128, 128, 64, 321, [200], "f32"), (2, 8, 64, 128, 64, 2048, [1000, 2048], "bf16")])
def test_in_place_with_more_segments_than_fit_at_once(B, G, H, N, P, T, lens, io):
    """Two to four segments a row, more workgroups than the GPU holds, rows that
    end before their last segment: no segment may start from what another one
    has already written.  All heads against the call out of place, some heads
    against the 64-bit form."""
    require_gpu()
    announce(f"ssm in place B={B} G={G} H={H} N={N} P={P} T={T} lens={lens} io={io}")
    d, s0 = inputs(12, B, T, G, H, N, P, io)
    apart = prefill(d, s0, G, lens)
    got = prefill(d, s0, G, lens, in_place=True)
    # Both are off by ssm_units of the sum of magnitudes at most, in bf16 by the
    # roundings of `check` besides.  The magnitudes: the scan of absolute values.
    mag, M = prefill(dict(d, x=d["x"].abs().float(), b=d["b"].abs().float(), c=d["c"].abs().float(),
                          D=d["D"].abs()), s0.abs(), G, lens)
    unit = ref.ssm_units(T, N) * EPS
    bound = 2 * unit * mag + (2.0 ** -6 * mag if io == "bf16" else 0) + 1e-30
    for b, n in enumerate(ref.clip_lens(lens, B, T)):
        assert ref.worst(got[0][b, :n], apart[0][b, :n].double(), bound[b, :n]) <= 1
        assert (got[0][b, n:] == 7).all()
    assert ref.worst(got[1], apart[1].double(), 2 * unit * M + 1e-30) <= 1
    heads, g = list(range(0, H, 16)), H // G
    for b, n in enumerate(ref.clip_lens(lens, B, T)):
        n = min(n, 450)                      # the 64-bit form's share of a long row
        part = dict(d, **{k: d[k][b: b + 1, :n, heads] for k in ("x", "dt")},
                    **{k: d[k][b: b + 1, :n, [h // g for h in heads]] for k in ("b", "c")},
                    **{k: d[k][heads] for k in ("A_log", "dt_bias", "D")})
        want, m, S, Ms = ref.ssm(**part, state=s0[b: b + 1, heads])
        bd = unit * m + (2.0 ** -8 * (want.abs() + m) if io == "bf16" else 0) + 1e-30
        assert ref.worst(got[0][b: b + 1, :n, heads], want, bd) <= 1
        if n == ref.clip_lens(lens, B, T)[b]:
            assert ref.worst(got[1][b: b + 1, heads], S, unit * Ms + 1e-30) <= 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 8, 100, 500])
def test_rates_past_the_largest_float(T, io):
    """exp(A_log) of 2^128 and more: a token forgets everything before it, one with
    a step size of 0 nothing.  Steps, the walk, chunks and segments agree."""
    require_gpu()
    announce(f"ssm rates past fp32 T={T} io={io}")
    d, s0 = inputs(14, 2, T, 1, 4, 32, 32, io)
    d["A_log"] = torch.tensor([88.8, 100.0, 1e4, 60.0])   # in 64 bits the third is infinite, too
    d["dt"][:, ::3] = -math.inf
    d["dt"][1, T // 2] = 4.0
    lens = [T, (T + 1) // 2]
    # The form takes the rate as it is; 1e4 stands for any that is as good as infinite.
    known = dict(d, A_log=d["A_log"].clamp(max=700.0))
    check(known, s0, prefill(d, s0, 1, lens), lens)
    g, S = up(d), s0.to(DEV)
    y, ys = torch.empty((2, 4, 32), dtype=g["x"].dtype, device=DEV), []
    for t in range(min(T, 8)):
        xbc = torch.cat([g[k][:, t].flatten(1) for k in ("x", "b", "c")], 1).contiguous()
        gdr.gdr_ssm_step(xbc, g["dt"][:, t].contiguous(), g["A_log"], g["dt_bias"], g["D"], S, y,
                         G=1, H=4, N=32, P=32)
        ys.append(y.cpu())
    cut = {k: v[:, :len(ys)] if k in ("x", "b", "c", "dt") else v for k, v in known.items()}
    check(cut, s0, (torch.stack(ys, 1), S.cpu()))


def test_differences_behind_an_enormous_decay_stay_exact():
    """A step size of 1e30 in a chunk: the tokens behind it decay as without it."""
    require_gpu()
    announce("ssm enormous step size inside a chunk")
    d, s0 = inputs(15, 1, 200, 1, 2, 16, 32, "f32")
    d["dt"][0, [5, 70, 130]] = 1e30
    d["x"][0, [5, 70, 130]] = 0.0                          # ... that writes nothing
    check(d, s0, prefill(d, s0, 1))


@pytest.mark.parametrize("T,N,P,strong", [(100, 16, 32, True), (100, 128, 64, True),
                                          (70, 16, 64, False), (130, 32, 128, True)])
def test_bf16_outputs_round_once(T, N, P, strong):
    """bf16 outputs of the chunks against the 64-bit form rounded once: a chunk's
    weights and the state lose 2^-15 of themselves on their way into the products,
    and a term is off by ssm_units of 2^-24 as in fp32."""
    require_gpu()
    announce(f"ssm, one rounding T={T} N={N} P={P} strong={strong}")
    d, s0 = inputs(16, 2, T, 2, 4, N, P, "bf16", strong=strong)
    d["D"] = None
    y, _ = prefill(d, s0, 2)
    want, mag, _, _ = ref.ssm(**d, state=s0)
    close = (2.0 ** -15 + ref.ssm_units(T, N) * EPS) * mag
    assert ref.worst(y, want, 2.0 ** -8 * (want.abs() + close) + close + 1e-30) <= 1
    # That leaves a difference only where a tie between two bf16 values lies within
    # `close`: for 2 close / step of the values, a step each.  The step is 2^-7 of a
    # value at most, so the mean square of the difference is at most
    # 2 close 2^-7 |value|.
    once = want.to(torch.bfloat16).double()
    assert ((y.double() - once) ** 2).mean() <= (2.0 ** -6 * close * (want.abs() + close)).mean()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [8, 9, 100])
def test_small_and_large_step_sizes(T, io):
    """softplus from -85 to 85, one step size a head: the other tokens' are 0, so the
    state is d B x, off by the softplus (8 units), the weight, its product with x and
    that with B (4).  In steps and walks (up to 8 tokens) e^z comes from a product
    with log2(e) that rounds before the exp2, as does the constant: 1.25 |z| units."""
    require_gpu()
    announce(f"ssm step sizes over the range T={T} io={io}")
    zs = [-85.0, -70.3, -52.7, -33.1, -20.9, -9.77, -3.3, -0.51, 0.0, 0.3, 2.9, 7.7, 15.9, 31.0,
          60.4, 85.0]
    H = len(zs)
    d, _ = inputs(17, 1, T, 1, H, 16, 16, io)
    d["dt"][:] = -math.inf
    d["dt"][0, T - 2] = torch.tensor(zs)
    d["dt_bias"] = d["D"] = None
    _, s = prefill(d, None, 1)
    z = torch.tensor(zs).double()
    step = torch.where(z > 30, z, torch.log1p(torch.exp(z.clamp(max=30))))
    want = step[:, None, None] * d["b"][0, T - 2, 0].double()[None, :, None] \
        * d["x"][0, T - 2].double()[:, None, :]
    walk = 12 + 1.25 * z.abs()[:, None, None]
    units = walk if T <= 8 else 12
    assert ref.worst(s[0], want, units * EPS * want.abs() + 1e-37) <= 1
    g, S = up(d), torch.zeros(1, H, 16, 16, device=DEV)
    xbc = torch.cat([g[k][:, T - 2].flatten(1) for k in ("x", "b", "c")], 1).contiguous()
    gdr.gdr_ssm_step(xbc, g["dt"][:, T - 2].contiguous(), g["A_log"], None, None, S,
                     torch.empty((1, H, 16), dtype=xbc.dtype, device=DEV), G=1, H=H, N=16, P=16)
    assert ref.worst(S[0].cpu(), want, walk * EPS * want.abs() + 1e-37) <= 1
