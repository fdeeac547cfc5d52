"""Plain 64-bit forms of the layers beside the gated delta rule, on the CPU, and
the bounds their kernels are held to.

Each form returns the result and its magnitude: the same sum with every term
taken absolutely, which is what roundings inside the sum scale with.  A
rounding to a type is off by at most half a step (HALF), relative to the value.
"""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F64 = torch.float64


def clip_lens(lens, B, T):
    return [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens]


def conv(x, weight, bias, state, silu=True, lens=None):
    """x [B,T,C], state [B,W-1,C] or None -> y (0 behind a row's end), |y| bound, state."""
    B, T, C = x.shape
    W = weight.shape[1]
    x, w = x.to(F64), weight.to(F64)
    s = torch.zeros(B, W - 1, C, dtype=F64) if state is None else state.to(F64)
    seen = torch.cat([s, x], 1)
    y, mag = torch.zeros(B, T, C, dtype=F64), torch.zeros(B, T, C, dtype=F64)
    if bias is not None:
        y, mag = y + bias.to(F64), mag + bias.to(F64).abs()
    for i in range(W):
        y = y + w[:, i] * seen[:, i: i + T]
        mag = mag + (w[:, i] * seen[:, i: i + T]).abs()
    if silu:
        y = y / (1 + torch.exp(-y))
    n = clip_lens(lens, B, T)
    return y, mag, torch.stack([seen[b, k: k + W - 1] for b, k in enumerate(n)])


def conv_bound(ref, mag, dtype, W):
    # W + 1 additions and products, then the sigmoid's exp2, sum, reciprocal
    # and product: SiLU's slope is at most 1.1, and its own chain is off by
    # (1.45 |s| + 6) units at most, |s| <= mag.
    units = 2 * (W + 1) + 8 + 1.5 * mag
    return HALF[dtype] * ref.abs() + units * 2.0 ** -24 * mag + 1e-30


def ssm(x, b, c, dt, A_log, dt_bias, D, state, lens=None):
    """Token by token.  x [B,T,H,P], b, c [B,T,G,N], dt [B,T,H], state
    [B,H,N,P] or None -> y, |y|, state, |state|."""
    B, T, H, P = x.shape
    G, N = b.shape[2:]
    x, b, c = x.to(F64), b.to(F64), c.to(F64)
    rate = torch.exp(A_log.to(F64))
    z = dt.to(F64) + (0 if dt_bias is None else dt_bias.to(F64))
    d = torch.where(z > 30, z, torch.log1p(torch.exp(z.clamp(max=30))))
    a = torch.exp(-rate * d)
    skip = torch.zeros(H, dtype=F64) if D is None else D.to(F64)
    S = torch.zeros(B, H, N, P, dtype=F64) if state is None else state.to(F64).clone()
    M = S.abs()
    y, mag = torch.zeros(B, T, H, P, dtype=F64), torch.zeros(B, T, H, P, dtype=F64)
    n = clip_lens(lens, B, T)
    for t in range(T):
        on = torch.tensor([t < k for k in n])
        if not on.any():
            break
        bt = b[:, t].repeat_interleave(H // G, 1)
        ct = c[:, t].repeat_interleave(H // G, 1)
        add = (d[:, t, :, None] * bt)[..., None] * x[:, t, :, None, :]
        S[on] = (a[:, t, :, None, None] * S + add)[on]
        M[on] = (a[:, t, :, None, None] * M + add.abs())[on]
        y[on, t] = ((S * ct[..., None]).sum(2) + skip[:, None] * x[:, t])[on]
        mag[on, t] = ((M * ct.abs()[..., None]).sum(2) + (skip[:, None] * x[:, t]).abs())[on]
    return y, mag, S, M


def ssm_units(T, N):
    """Units of 2^-24 a term of y or S may be off by: a token's decay, product
    and sum round at most 4 times, so a term of age t is off by 4 t; the read
    sums N rows; the token's own step size, weight and gate add 16."""
    return 4 * T + N + 16


def ssm_norm(T, N):
    """The same over a whole tensor, by 2-norm.  A token's decay is shared by all
    elements of a state, so its rounding does not average out over them: with
    `units` independent roundings, each uniform over half a step, the sum has a
    standard deviation of sqrt(units / 3) half steps; three of those."""
    return math.sqrt(3 * ssm_units(T, N)) * 2.0 ** -24


def e4m3(v):
    """Nearest e4m3 value (ties to even significands), by the spacing of its binade."""
    nan = torch.isnan(v)
    v = torch.nan_to_num(v, nan=0.0, posinf=448.0, neginf=-448.0).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(nan, torch.nan, torch.round(v / step) * step)


def pow2_scale(x):
    """Smallest 2^k >= 2^-100 with max|finite x| <= 448 * 2^k."""
    top = x[torch.isfinite(x)].abs().max().item() if torch.isfinite(x).any() else 0.0
    k = -100
    while top > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append(k, v, kc, vc, ks, vs, table, pos, lens=None):
    """Caches as values of codes (F64), [pages,H,page,D] and [pages,H,D,page]; all
    four are updated in place."""
    B, T, H, D = k.shape
    pages, page = kc.shape[0], kc.shape[2]
    n = clip_lens(lens, B, T)
    for b in range(B):
        p = int(pos[b])
        for at in range(table.shape[1]):
            new = [t for t in range(n[b]) if p + t >= 0 and (p + t) // page == at]
            pg = int(table[b, at])
            if not new or not 0 <= pg < pages:
                continue
            had = max(0, p - at * page)
            slots = [p + t - at * page for t in new]
            for x, cache, scale in ((k, kc, ks), (v, vc.transpose(2, 3), vs)):
                for h in range(H):
                    rows = x[b, new, h].to(F64)
                    s = pow2_scale(rows)
                    if had:
                        s = max(s, float(scale[pg, h]))
                        cache[pg, h, :had] = e4m3(cache[pg, h, :had] * (float(scale[pg, h]) / s))
                    cache[pg, h, slots] = e4m3(rows / s)
                    scale[pg, h] = s


def attention(q, kc, vc, ks, vs, table, pos, scale, lens=None):
    """q [B,T,Hq,D]; caches as values of codes (F64) -> o, sum of p |v|, the
    largest |score| of a row."""
    B, T, Hq, D = q.shape
    pages, H, page = kc.shape[:3]
    n = clip_lens(lens, B, T)
    o, mag = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    top = torch.zeros(B, T, Hq, dtype=F64)
    for b in range(B):
        cap = table.shape[1] * page
        for t in range(n[b]):
            last = min(int(pos[b]) + t + 1, cap)
            keys = [j for j in range(max(last, 0)) if 0 <= int(table[b, j // page]) < pages]
            if not keys:
                continue
            pg = torch.tensor([int(table[b, j // page]) for j in keys])
            sl = torch.tensor([j % page for j in keys])
            for h in range(Hq):
                g = h // (Hq // H)
                K = kc[pg, g, sl] * ks.to(F64)[pg, g][:, None]
                V = vc[pg, g, :, sl] * vs.to(F64)[pg, g][:, None]
                qh = q[b, t, h].to(F64)
                z = (K @ qh) * scale
                p = torch.softmax(z, 0)
                o[b, t, h], mag[b, t, h] = p @ V, p @ V.abs()
                top[b, t, h] = ((K.abs() @ qh.abs()) * abs(scale)).max()
    return o, mag, top


def rel(x, ref):
    d = (x.to(F64) - ref).norm().item()
    return d / ref.norm().item() if ref.norm().item() else d


def worst(x, ref, bound):
    """Largest error in units of its bound (NaN counts as infinite)."""
    r = ((x.to(F64) - ref).abs() / bound)
    return math.inf if torch.isnan(r).any() else float(r.max()) if r.numel() else 0.0
