"""The 8-bit key/value cache on the GPU: writes against their 64-bit form, code
for code, and attention over it."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from tests import layer_ref as ref
from tests.gpu_util import DEV, announce, io_dtype, require_gpu

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


class Cache:
    """A pool on the device and the same on the host in 64 bits."""

    def __init__(self, seed, B, per, Hkv, D, page, spare=3):
        gen = torch.Generator().manual_seed(seed)
        self.pages, self.page, self.per = B * per + spare, page, per
        self.table = torch.randperm(self.pages, generator=gen)[: B * per].view(B, per).to(torch.int32)
        size = torch.exp(torch.randn(self.pages, Hkv, 1, 1, generator=gen) * 0.7)
        for n, shape in (("k", (Hkv, page, D)), ("v", (Hkv, D, page))):
            x = torch.randn(self.pages, *shape, generator=gen) * size
            s = torch.tensor([[ref.pow2_scale(x[p, h]) for h in range(Hkv)]
                              for p in range(self.pages)], dtype=torch.float32)
            setattr(self, n + "c", ref.e4m3(x.double() / s.double()[..., None, None]))
            setattr(self, n + "s", s)

    def device(self):
        return (self.kc.to(F8).to(DEV), self.vc.to(F8).to(DEV), self.ks.to(DEV), self.vs.to(DEV))

    def host(self):
        return self.kc.clone(), self.vc.clone(), self.ks.clone().double(), self.vs.clone().double()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def same(got, want):
    a, b = got.cpu().double(), want.double()
    assert a.shape == b.shape
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def append(c, k, v, pos, lens=None, dev=None):
    dev = dev or c.device()
    gdr.gdr_kv_append(k.to(DEV), v.to(DEV), *dev, c.table.to(DEV), i32(pos),
                      lens=None if lens is None else i32(lens))
    return dev


# ---------------------------------------------------------------------------
# writes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 16), (2, 128, 64), (3, 64, 128), (5, 128, 32)])
@pytest.mark.parametrize("T", [1, 2, 8, 15, 33, 130])
def test_append(T, Hkv, D, page, io):
    require_gpu()
    announce(f"append T={T} Hkv={Hkv} D={D} page={page} io={io}")
    B, per = 4, -(-(T + 150) // page)
    c = Cache(T + page, B, per, Hkv, D, page)
    gen = torch.Generator().manual_seed(T)
    # small and large new values: scales that stay and scales that grow
    size = torch.tensor([0.05, 1.0, 30.0, 4.0])[:, None, None, None]
    k = (torch.randn(B, T, Hkv, D, generator=gen) * size).to(io_dtype(io))
    v = (torch.randn(B, T, Hkv, D, generator=gen) * size.flip(0)).to(io_dtype(io))
    for pos, lens in (([0, 1, page - 1, 150], None), ([page, 77, 2 * page - 1, 149], [T, 1, T // 2, T]),
                      ([-3, -T, 5, per * page - 1], [T, T, 0, T])):
        want = c.host()
        ref.append(k, v, *want, c.table, pos, lens)
        got = append(c, k, v, pos, lens)
        for a, b in zip(got, want):
            same(a, b)


def test_append_one_by_one_and_the_last_slot():
    """A page filled token by token, its scale growing: codes shift exactly."""
    require_gpu()
    announce("append token by token")
    c = Cache(3, 2, 3, 2, 64, 16)
    want, dev = c.host(), c.device()
    gen = torch.Generator().manual_seed(4)
    for t in range(40):
        k, v = (torch.randn(2, 1, 2, 64, generator=gen) * 1.3 ** t for _ in range(2))
        pos = [t, t + 8]
        ref.append(k, v, *want, c.table, pos)
        append(c, k, v, pos, dev=dev)
        for a, b in zip(dev, want):
            same(a, b)


def test_append_values_that_are_not_finite_zero_or_tiny():
    require_gpu()
    announce("append inf, NaN, zeros, subnormals, bounds of the scale")
    c = Cache(5, 6, 1, 1, 64, 16)
    x = torch.randn(6, 3, 1, 64)
    x[0, 1, 0, 3], x[0, 1, 0, 4], x[0, 2, 0, 5] = math.inf, -math.inf, math.nan
    x[1] = 0.0
    x[2] = x[2] * 1e-42
    x[3] = 448.0
    x[4] = 448.0 * (1 + 2.0 ** -23)
    x[5] = 3e38
    want = c.host()
    ref.append(x, -x, *want, c.table, [0] * 6)
    got = append(c, x, -x, [0] * 6)
    for a, b in zip(got, want):
        same(a, b)
    x[:] = math.nan
    want = c.host()
    ref.append(x, x, *want, c.table, [4] * 6)
    got = append(c, x, x, [4] * 6)
    for a, b in zip(got, want):
        same(a, b)


def test_append_does_not_follow_bad_pages():
    require_gpu()
    announce("append with page numbers outside the pool")
    c = Cache(6, 3, 4, 2, 64, 16)
    c.table[0, 1], c.table[1, 0], c.table[2, 2] = -1, c.pages, 2 ** 31 - 1
    k = torch.randn(3, 50, 2, 64)
    want = c.host()
    ref.append(k, -k, *want, c.table, [3, 0, 10])
    got = append(c, k, -k, [3, 0, 10])
    for a, b in zip(got, want):
        same(a, b)


@pytest.mark.parametrize("T", [2, 8, 9, 33])
@pytest.mark.parametrize("lens", [None, 0])
def test_append_far_in_front_of_the_sequence_writes_nothing(T, lens):
    """Positions near -2^31 (a sentinel for an idle row) are not followed."""
    require_gpu()
    announce(f"append at positions near -2^31 T={T} lens={lens}")
    c = Cache(17, 4, 4, 2, 64, 16)
    k = torch.randn(4, T, 2, 64)
    pos = [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + T, -T]
    want = c.host()
    got = append(c, k, -k, pos, None if lens is None else [lens] * 4)
    for a, b in zip(got, want):
        same(a, b)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attend(c, q, pos, scale, lens=None, dev=None, table=None, fill=7.0):
    B, T, Hq, D = q.shape
    dev = dev or c.device()
    table = c.table if table is None else table
    n = gdr.gdr_attn_workspace_size(B, T, Hq, dev[0].shape[1], D, c.page, table.shape[1], q.dtype)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None
    o = torch.full(q.shape, fill, dtype=q.dtype, device=DEV)
    gdr.gdr_attn_cached(q.to(DEV), *dev, table.to(DEV), i32(pos), o, ws, scale=scale,
                        lens=None if lens is None else i32(lens))
    torch.cuda.synchronize()
    return o.cpu()


def check(c, q, o, pos, scale, lens=None, table=None):
    table = c.table if table is None else table
    want, mag, top = ref.attention(q, c.kc, c.vc, c.ks, c.vs, table, pos, scale, lens)
    # A score sums D products (D + 4 roundings) of magnitude `top` and goes
    # through exp2 (its argument rounds twice more); a probability and its
    # value add the roundings of p, of the product and of the running sums.
    keys = max(1, max(p for p in pos) + q.shape[1])
    units = (q.shape[-1] + 8) * top[..., None] + keys ** 0.5 * 4 + 32
    bound = units * 2.0 ** -24 * mag + 1e-30
    if q.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + mag)   # the output's rounding, and p's own
    for b, n in enumerate(ref.clip_lens(lens, *q.shape[:2])):
        assert ref.worst(o[b, :n], want[b, :n], bound[b, :n]) <= 1
        assert (o[b, n:] == 7).all()
    keep = torch.tensor([[t < n for t in range(q.shape[1])]
                         for n in ref.clip_lens(lens, *q.shape[:2])])
    if keep.any() and want[keep].norm() > 0:
        assert ref.rel(o[keep], want[keep]) <= (2.0 ** -8 if q.dtype == torch.bfloat16 else 5e-6)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,page,ctx", [
    (1, 1, 1, 1, 64, 16, 0), (3, 1, 4, 2, 128, 64, 63), (2, 1, 8, 1, 64, 32, 64),
    (4, 1, 7, 1, 128, 16, 100), (2, 1, 40, 2, 64, 128, 300), (1, 1, 32, 8, 128, 64, 700),
    (2, 2, 6, 3, 64, 16, 31), (1, 5, 8, 2, 128, 32, 200), (3, 17, 4, 4, 64, 64, 90),
    (2, 40, 2, 1, 128, 128, 50), (1, 130, 3, 1, 64, 16, 77), (2, 65, 14, 2, 64, 32, 0)])
def test_attention(B, T, Hq, Hkv, D, page, ctx, io):
    require_gpu()
    announce(f"attention B={B} T={T} Hq={Hq} Hkv={Hkv} D={D} page={page} ctx={ctx} io={io}")
    c = Cache(ctx + T, B, -(-(ctx + T + 3) // page), Hkv, D, page)
    gen = torch.Generator().manual_seed(ctx)
    q = torch.randn(B, T, Hq, D, generator=gen).to(io_dtype(io))
    pos = [max(0, ctx - 13 * i) for i in range(B)]
    s = 1 / math.sqrt(D)
    check(c, q, attend(c, q, pos, s), pos, s)
    lens = [max(0, T - 1), T + 4, -2, 1][:B]
    check(c, q, attend(c, q, pos, s, lens), pos, s, lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_queries_with_nothing_to_attend_to(T, io):
    """Positions before the sequence, pages outside the pool, no pages at all."""
    require_gpu()
    announce(f"attention over nothing T={T} io={io}")
    c = Cache(8, 4, 6, 2, 64, 16)
    q = torch.randn(4, T, 4, 64).to(io_dtype(io))
    pos = [-T, -1, 2, 60]
    table = c.table.clone()
    table[2] = -1
    table[3, 0], table[3, 2] = c.pages + 5, -7
    o = attend(c, q, pos, 0.125, table=table)
    check(c, q, o, pos, 0.125, table=table)
    assert (o[0] == 0).all() and (o[2] == 0).all()
    assert (attend(c, q, pos, 0.125, table=table[:, :0].contiguous()) == 0).all()
    pos = [95 - T, 96, 97, 2 ** 31 - 1]                  # up to and past the table's end
    pos_ref = [95 - T, 96, 97, 96]
    check(c, q, attend(c, q, pos, 0.125), pos_ref, 0.125)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 20])
def test_nan_codes_behind_the_last_position_do_not_matter(T, io):
    require_gpu()
    announce(f"attention with NaN codes behind the end T={T} io={io}")
    c = Cache(9, 2, 8, 2, 128, 32)
    q = torch.randn(2, T, 8, 128).to(io_dtype(io))
    pos = [70, 101]
    clean = attend(c, q, pos, 0.09)
    dev = c.device()
    for b in range(2):
        end = pos[b] + T
        for j in range(8):
            pg, n = int(c.table[b, j]), min(max(end - 32 * j, 0), 32)
            dev[0].view(torch.uint8)[pg, :, n:] = 0x7F
            dev[1].view(torch.uint8)[pg, :, :, n:] = 0xFF
            if n == 0:
                dev[2][pg], dev[3][pg] = math.nan, math.inf
    assert torch.equal(attend(c, q, pos, 0.09, dev=dev), clean)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_large_scores_and_scales(io):
    """Scores of several hundred, and pages whose value scales differ by 2^40."""
    require_gpu()
    announce(f"attention with large scores io={io}")
    c = Cache(10, 2, 5, 1, 64, 64)
    c.ks *= 16
    c.vs[::2] *= 2.0 ** 40
    q = (torch.randn(2, 1, 4, 64) * 4).to(io_dtype(io))
    pos = [299, 130]
    o = attend(c, q, pos, 0.125)
    want, mag, top = ref.attention(q, c.kc, c.vc, c.ks, c.vs, c.table, pos, 0.125)
    bound = ((72 * top[..., None] + 128) * 2.0 ** -24 + (2.0 ** -7 if io == "bf16" else 0)) * mag
    assert ref.worst(o, want, bound) <= 1


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_all_keys_alike_gives_the_mean(io):
    require_gpu()
    announce(f"attention over equal keys io={io}")
    c = Cache(11, 1, 20, 1, 64, 64)
    c.kc[:] = 0
    q = torch.randn(1, 1, 16, 64).to(io_dtype(io))
    pos = [1200]
    check(c, q, attend(c, q, pos, 1.0), pos, 1.0)


def test_pages_shared_by_rows():
    """Rows that start with the same pages (a common prefix) read them together."""
    require_gpu()
    announce("attention over shared pages")
    c = Cache(12, 3, 4, 2, 128, 16)
    c.table[1, :2] = c.table[0, :2]
    c.table[2, :3] = c.table[0, :3]
    q = torch.randn(3, 4, 4, 128).to(torch.bfloat16)
    pos = [50, 44, 59]
    check(c, q, attend(c, q, pos, 0.1), pos, 0.1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,T", [(4, 6), (2, 100)])
def test_nan_token_does_not_reach_earlier_queries(Hq, T, io):
    """A new token whose key or value holds NaN: queries before it do not see it."""
    require_gpu()
    announce(f"attention with a NaN token Hq={Hq} T={T} io={io}")
    c = Cache(13, 2, 12, 2, 64, 16)
    q = torch.randn(2, T, Hq, 64).to(io_dtype(io))
    pos = [37, 64]
    clean = attend(c, q, pos, 0.125)
    at = T // 2
    for b in range(2):
        p = pos[b] + at
        pg, sl = int(c.table[b, p // 16]), p % 16
        c.vc[pg, 0, 7, sl] = math.nan                    # head 0: one column of the value
        c.kc[pg, 1, sl, 3] = math.nan                    # head 1: the key
    o = attend(c, q, pos, 0.125)
    half = Hq // 2
    assert torch.equal(o[:, :at], clean[:, :at])
    cols = [d for d in range(64) if d != 7]
    assert torch.equal(o[:, :, :half][..., cols], clean[:, :, :half][..., cols])
    assert torch.isnan(o[:, at:, :half, 7]).all() and torch.isnan(o[:, at:, half:]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_score_scales(scale, T, io):
    """Negative, zero (the mean of the values in sight) and large score scales."""
    require_gpu()
    announce(f"attention with scale {scale} T={T} io={io}")
    c = Cache(14, 2, 14, 1, 64, 16)
    q = torch.randn(2, T, 2, 64).to(io_dtype(io))
    pos = [90, 131]
    check(c, q, attend(c, q, pos, scale), pos, scale)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_table_in_many_splits(io):
    """One request with room for many more keys than it has, and one that uses them."""
    require_gpu()
    announce(f"attention over a long table io={io}")
    c = Cache(15, 2, 160, 1, 64, 64)
    q = torch.randn(2, 1, 2, 64).to(io_dtype(io))
    pos = [20, 10200]
    check(c, q, attend(c, q, pos, 0.125), pos, 0.125)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (64, 128)])
@pytest.mark.parametrize("T", [1, 20, 70])
def test_pages_outside_the_pool_count_for_nothing(T, D, page, io):
    """Holes in the table among keys that every query sees; the pool's first page,
    which no row names, holds NaN codes and scales that are not finite."""
    require_gpu()
    announce(f"attention with holes in the table T={T} D={D} page={page} io={io}")
    B, keys = 2, 512 + T
    c = Cache(16, B, -(-keys // page), 2, D, page)
    c.table[c.table == 0] = next(p for p in range(1, c.pages) if not (c.table == p).any())
    c.table[0, 0], c.table[1, 192 // page], c.table[1, 320 // page] = -1, c.pages, 2 ** 31 - 1
    q = torch.randn(B, T, 4, D, generator=torch.Generator().manual_seed(T)).to(io_dtype(io))
    pos, scale = [512, 400], 1 / math.sqrt(D)
    clean = attend(c, q, pos, scale)
    check(c, q, clean, pos, scale)
    for ks, vs in ((math.nan, math.nan), (math.inf, math.inf)):
        dev = c.device()
        dev[0].view(torch.uint8)[0], dev[1].view(torch.uint8)[0] = 0x7F, 0xFF
        dev[2][0], dev[3][0] = ks, vs
        assert torch.equal(attend(c, q, pos, scale, dev=dev), clean)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 70])
@pytest.mark.parametrize("at", [5, 69])
def test_nan_value_of_a_key_that_hardly_counts(at, T, io):
    """NaN times a probability is NaN however small that is: past fp32's range, and
    so with a value scale of 2^-100."""
    require_gpu()
    announce(f"attention, NaN value of a far key at={at} T={T} io={io}")
    c = Cache(18, 2, 10, 1, 64, 16)
    q = torch.randn(2, T, 4, 64).to(io_dtype(io))
    q[..., 0] = 30.0
    pos = [69, 80]
    for b, k in ((0, -96.0), (1, -10.0)):               # p about e^-288, and e^-30 2^-100
        pg = int(c.table[b, at // 16])
        c.ks[pg], c.kc[pg, 0] = 1.0, 0.0
        c.kc[pg, 0, at % 16, 0] = k
        c.vc[pg, 0, 11, at % 16] = math.nan
        if b == 1:
            c.vs[pg] = 2.0 ** -100
    o = attend(c, q, pos, 0.1)
    assert torch.isnan(o[..., 11]).all()
    assert torch.isfinite(o[..., [d for d in range(64) if d != 11]]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("scale", [math.nan, math.inf])
def test_score_scale_that_is_not_finite(scale, T, io):
    """Scores of NaN, or of infinities and NaN: no finite answer, in either kernel;
    queries with nothing to attend to still give zeros."""
    require_gpu()
    announce(f"attention with scale {scale} T={T} io={io}")
    c = Cache(19, 2, 14, 1, 64, 16)
    q = torch.randn(2, T, 2, 64).to(io_dtype(io))
    o = attend(c, q, [90, -T], scale)
    assert torch.isnan(o[0]).all() and (o[1] == 0).all()


@pytest.mark.parametrize("T,Hq,D,page", [(1, 8, 64, 16), (40, 8, 128, 32), (150, 4, 64, 64),
                                         (150, 8, 128, 16)])
def test_bf16_outputs_round_once(T, Hq, D, page):
    """bf16 outputs against the 64-bit form rounded once.  Scores are single exact
    products, so what is off before the output's rounding is what p loses (2^-15 of
    it), and fp32's units: the score's factor, product and difference at |z| log2(e)
    <= 16 (48), exp2, p and the sums (32 + 4 sqrt(keys))."""
    require_gpu()
    announce(f"attention, one rounding T={T} Hq={Hq} D={D} page={page}")
    gen = torch.Generator().manual_seed(T)
    c = Cache(20, 1, -(-(300 + T) // page), 2, D, page)
    c.ks[:], c.kc = 1.0, ref.e4m3(2 * torch.randn(c.kc.shape, generator=gen, dtype=torch.float64))
    q = torch.zeros(1, T, Hq, D, dtype=torch.bfloat16)
    q[0, :, :, torch.randperm(D, generator=gen)[0]] = 1.0
    o = attend(c, q, [300], 1.0)
    want, mag, top = ref.attention(q, c.kc, c.vc, c.ks, c.vs, c.table, [300], 1.0)
    assert top.max() < 11
    close = (2.0 ** -15 + (80 + 4 * (300 + T) ** 0.5) * 2.0 ** -24) * mag
    assert ref.worst(o, want, 2.0 ** -8 * (want.abs() + close) + close + 1e-30) <= 1
    # That leaves a difference only where a tie between two bf16 values lies within
    # `close`: for 2 close / step of the values, a step each.  The step is 2^-7 of a
    # value at most, so the mean square of the difference is at most
    # 2 close 2^-7 |value|.
    once = want.to(torch.bfloat16).double()
    assert ((o.double() - once) ** 2).mean() <= (2.0 ** -6 * close * (want.abs() + close)).mean()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,page,ctx", [
    (29, 1, 5, 5, 128, 16, 1029), (10, 1, 12, 3, 64, 16, 2100), (3, 9, 2, 1, 64, 64, 1500)])
def test_many_steps_a_wave(B, T, Hq, Hkv, D, page, ctx, io):
    """Rows of many steps each, few and several query rows, large value scales: what
    one step leaves in a wave's registers does not reach the next step's scores."""
    require_gpu()
    announce(f"attention of many steps B={B} T={T} Hq={Hq} Hkv={Hkv} D={D} page={page} io={io}")
    c = Cache(21, B, -(-(ctx + T) // page), Hkv, D, page)
    c.vs *= 2.0 ** 16
    q = torch.randn(B, T, Hq, D, generator=torch.Generator().manual_seed(B)).to(io_dtype(io))
    pos = [ctx - (53 * i) % (ctx // 2) for i in range(B)]
    check(c, q, attend(c, q, pos, 1 / math.sqrt(D)), pos, 1 / math.sqrt(D))
