"""The layers together, as a model calls them: a prompt, then tokens one by one,
through convolution -> gated delta rule, convolution -> scan, and cache write ->
attention; the same captured in a graph and replayed; and on other streams."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
import oracle
from tests import layer_ref as ref
from tests.gpu_util import DEV, announce, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(gen, *s):
    return torch.randn(*s, generator=gen)


class Delta:
    """Convolution, then the gated delta rule (scalar gate)."""
    Hq, Hv, dk, dv, W = 2, 4, 32, 64, 4

    def __init__(self, gen, B):
        self.B = B
        self.widths = (self.Hq * self.dk, self.Hq * self.dk, self.Hv * self.dv)
        C = sum(self.widths)
        self.w, self.bias = (rnd(gen, C, self.W) * 0.6).to(DEV), (rnd(gen, C) * 0.2).to(DEV)
        self.conv = torch.zeros(B, self.W - 1, C, dtype=BF, device=DEV)
        self.S = torch.zeros(B, self.Hv, self.dk, self.dv, device=DEV)
        self.kw = dict(H_qk=self.Hq, H_v=self.Hv, dk=self.dk, dv=self.dv,
                       gate=gdr.GDR_GATE_SCALAR, scale=1 / math.sqrt(self.dk))

    def prompt(self, x, g, beta):
        B, T = x.shape[:2]
        qkv = [torch.empty(B, T, c, dtype=BF, device=DEV) for c in self.widths]
        gdr.gdr_conv_prefill(x, self.w, self.bias, self.conv, self.conv, qkv)
        o = torch.empty(B, T, self.Hv, self.dv, dtype=BF, device=DEV)
        ws = torch.empty(gdr.gdr_prefill_workspace_size(B, T, self.Hq, self.Hv, self.dk, self.dv,
                                                        32, BF, gdr.GDR_GATE_SCALAR),
                         dtype=torch.uint8, device=DEV)
        gdr.gdr_prefill_chunked(*qkv, g, beta, self.S, self.S, o, ws, chunk=32, **self.kw)
        return o

    def token(self, x, g, beta):
        qkv = torch.empty_like(x)
        gdr.gdr_conv_step(x, self.w, self.bias, self.conv, qkv)
        o = torch.empty(self.B, self.Hv, self.dv, dtype=BF, device=DEV)
        gdr.gdr_decode_step(qkv, g, beta, self.S, o, **self.kw)
        return o


def test_convolution_then_delta_rule():
    require_gpu()
    announce("chain conv -> gated delta rule: prompt of 45, 5 tokens")
    gen = torch.Generator().manual_seed(1)
    B, T, n = 2, 45, 5
    m = Delta(gen, B)
    C = sum(m.widths)
    x = rnd(gen, B, T + n, C).to(BF)
    g, beta = -rnd(gen, B, T + n, m.Hv).abs() * 0.2, rnd(gen, B, T + n, m.Hv)
    xd, gd, bd = x.to(DEV), g.to(DEV), beta.to(DEV)
    os = [m.prompt(xd[:, :T].contiguous(), gd[:, :T].contiguous(), bd[:, :T].contiguous())]
    for t in range(T, T + n):
        os.append(m.token(xd[:, t], gd[:, t].contiguous(), bd[:, t].contiguous())[:, None])
    got = torch.cat(os, 1).cpu()
    y, _, _ = ref.conv(x, m.w.cpu(), m.bias.cpu(), None)
    y = y.to(BF).double()                       # the rows pass in bf16
    q, k, v = (t.reshape(B, T + n, -1, w).numpy() for t, w in
               zip(y.split(m.widths, -1), (m.dk, m.dk, m.dv)))
    o, S = oracle.sequence(q, k, v, gdr.GDR_GATE_SCALAR, g.numpy(), beta.numpy(), None,
                           scale=1 / math.sqrt(m.dk))
    assert ref.rel(got, torch.from_numpy(o)) < 2e-2
    assert ref.rel(m.S.cpu(), torch.from_numpy(S)) < 2e-2


class Scan:
    """Convolution, then the selective state space scan."""
    G, H, N, P, W = 2, 4, 32, 64, 4

    def __init__(self, gen, B):
        self.B, self.size = B, dict(G=self.G, H=self.H, N=self.N, P=self.P)
        self.widths = (self.H * self.P, self.G * self.N, self.G * self.N)
        C = sum(self.widths)
        self.w, self.bias = (rnd(gen, C, self.W) * 0.6).to(DEV), (rnd(gen, C) * 0.2).to(DEV)
        self.A_log = torch.log(1 + 15 * torch.rand(self.H, generator=gen)).to(DEV)
        self.db, self.D = (rnd(gen, self.H) - 3).to(DEV), rnd(gen, self.H).to(DEV)
        self.conv = torch.zeros(B, self.W - 1, C, dtype=BF, device=DEV)
        self.S = torch.zeros(B, self.H, self.N, self.P, device=DEV)

    def prompt(self, x, dt, lens=None):
        B, T = x.shape[:2]
        xbc = [torch.zeros(B, T, c, dtype=BF, device=DEV) for c in self.widths]
        gdr.gdr_conv_prefill(x, self.w, self.bias, self.conv, self.conv, xbc, lens=lens)
        y = torch.zeros(B, T, self.H * self.P, dtype=BF, device=DEV)
        n = gdr.gdr_ssm_workspace_size(B, T, io_dtype=BF, **self.size)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        gdr.gdr_ssm_prefill(*xbc, dt, self.A_log, self.db, self.D, self.S, self.S, y, ws, lens=lens,
                            **self.size)
        return y

    def token(self, x, dt):
        xbc = torch.empty(self.B, sum(self.widths), dtype=BF, device=DEV)
        gdr.gdr_conv_step(x, self.w, self.bias, self.conv, xbc)
        y = torch.empty(self.B, self.H, self.P, dtype=BF, device=DEV)
        gdr.gdr_ssm_step(xbc, dt, self.A_log, self.db, self.D, self.S, y, **self.size)
        return y.view(self.B, -1)


def test_convolution_then_scan_over_a_padded_batch():
    require_gpu()
    announce("chain conv -> scan: prompts of 150, 83 and 1, 4 tokens")
    gen = torch.Generator().manual_seed(2)
    B, T, n, lens = 3, 150, 4, [150, 83, 1]
    m = Scan(gen, B)
    C = sum(m.widths)
    # The rows of a projection: [x|B|C] beside a gate the convolution skips.
    row = rnd(gen, B, T + n, C + 40).to(BF).to(DEV)
    dt = rnd(gen, B, T + n, m.H).to(DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    y = m.prompt(row[:, :T].contiguous()[..., 40:], dt[:, :T].contiguous(), ln)
    ys = [m.token(row[:, T + i, 40:], dt[:, T + i].contiguous()) for i in range(n)]
    for b, k in enumerate(lens):
        at = list(range(k)) + list(range(T, T + n))
        x = row[b: b + 1, at, 40:].cpu()
        z, _, _ = ref.conv(x, m.w.cpu(), m.bias.cpu(), None)
        z = z.to(BF)
        xs, bs, cs = z.split(m.widths, -1)
        L = len(at)
        want, mag, S, M = ref.ssm(xs.reshape(1, L, m.H, m.P), bs.reshape(1, L, m.G, m.N),
                                  cs.reshape(1, L, m.G, m.N), dt[b: b + 1, at].cpu(),
                                  m.A_log.cpu(), m.db.cpu(), m.D.cpu(), None)
        got = torch.cat([y[b, :k].cpu()] + [t[b: b + 1].cpu() for t in ys]).view(1, L, m.H, m.P)
        # bf16 rows between the layers: one of them on the other side of a tie
        # moves a term by a full step (2^-7 of it).
        assert ref.worst(got, want, 2.0 ** -8 * (want.abs() + 3 * mag)) <= 1
        assert ref.rel(got, want) <= 2.0 ** -7
        assert ref.worst(m.S[b: b + 1].cpu(), S, 2.0 ** -7 * M + 1e-30) <= 1
        assert (y[b, k:] == 0).all()


class Attention:
    Hq, Hkv, D, page = 8, 2, 64, 16

    def __init__(self, gen, B, room):
        per = -(-room // self.page)
        n = B * per
        self.table = torch.randperm(n, generator=gen).view(B, per).to(torch.int32).to(DEV)
        self.kc = torch.zeros(n, self.Hkv, self.page, self.D, dtype=torch.uint8, device=DEV)
        self.vc = torch.zeros(n, self.Hkv, self.D, self.page, dtype=torch.uint8, device=DEV)
        self.ks, self.vs = (torch.zeros(n, self.Hkv, device=DEV) for _ in range(2))

    def run(self, q, k, v, pos, lens=None):
        gdr.gdr_kv_append(k, v, self.kc, self.vc, self.ks, self.vs, self.table, pos, lens=lens)
        B, T = q.shape[:2]
        n = gdr.gdr_attn_workspace_size(B, T, self.Hq, self.Hkv, self.D, self.page,
                                        self.table.shape[1], BF)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        o = torch.zeros_like(q)
        gdr.gdr_attn_cached(q, self.kc, self.vc, self.ks, self.vs, self.table, pos, o, ws,
                            scale=1 / math.sqrt(self.D), lens=lens)
        return o


def test_cache_write_then_attention():
    require_gpu()
    announce("chain append -> attention: prompts of 70 and 33, 6 tokens")
    gen = torch.Generator().manual_seed(3)
    B, T, n, lens = 2, 70, 6, [70, 33]
    m = Attention(gen, B, T + n)
    q = rnd(gen, B, T + n, m.Hq, m.D).to(BF)
    k, v = (rnd(gen, B, T + n, m.Hkv, m.D).to(BF) for _ in range(2))
    qd, kd, vd = (t.to(DEV) for t in (q, k, v))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    cut = lambda t: t[:, :T].contiguous()  # noqa: E731
    o = m.run(cut(qd), cut(kd), cut(vd), i32([0, 0]), i32(lens)).cpu()
    one = lambda t, i: t[:, T + i: T + i + 1].contiguous()  # noqa: E731
    os = [m.run(one(qd, i), one(kd, i), one(vd, i), i32([k0 + i for k0 in lens])).cpu()
          for i in range(n)]
    for b, k0 in enumerate(lens):
        at = list(range(k0)) + list(range(T, T + n))
        got = torch.cat([o[b, :k0]] + [t[b] for t in os])
        K, V = (t[b, at].double() for t in (k, v))
        assert (o[b, k0:] == 0).all()
        for i in range(len(at)):
            for h in range(m.Hq):
                p = torch.softmax(K[: i + 1, h // 4] @ q[b, at[i], h].double() / math.sqrt(m.D), 0)
                want = p @ V[: i + 1, h // 4]
                # e4m3 keeps values to 2^-4 of themselves: scores move by up to
                # 2^-4 sum|q k|/sqrt(D) in the worst case; as independent
                # roundings, uniform over half a step, by 2^-4/sqrt(3) of the
                # norm of their terms, times 5 for the largest of all.
                z = (K[: i + 1, h // 4] * q[b, at[i], h].double()).norm(dim=1).max() / math.sqrt(m.D)
                slack = 5 * 2.0 ** -4 / math.sqrt(3) * (1 + 2 * float(z))
                assert (got[i, h].double() - want).norm() <= slack * (p.norm() * V.norm(dim=1).max())


def test_graph_replays_match_eager():
    require_gpu()
    announce("graph: both chains and the cache, 3 replays")
    gen = torch.Generator().manual_seed(4)
    B, T = 2, 200
    a, s, c = Delta(gen, B), Scan(gen, B), Attention(gen, B, T + 4)
    xa, xs = rnd(gen, B, T, sum(a.widths)).to(BF).to(DEV), rnd(gen, B, T, sum(s.widths)).to(BF).to(DEV)
    g, beta, dt = (rnd(gen, B, T, 4).to(DEV) for _ in range(3))
    g = -g.abs() * 0.2
    q, k, v = (rnd(gen, B, T, h, 64).to(BF).to(DEV) for h in (8, 2, 2))
    pos = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    q1, k1, v1 = (t[:, :1].contiguous() for t in (q, k, v))
    pos1 = pos + T
    state = [a.conv, a.S, s.conv, s.S, c.kc, c.vc, c.ks, c.vs]
    start = [t.clone() for t in state]

    def work():
        return [a.prompt(xa, g, beta), a.token(xa[:, 0], g[:, 0].contiguous(), beta[:, 0].contiguous()),
                s.prompt(xs, dt), s.token(xs[:, 0], dt[:, 0].contiguous()),
                c.run(q, k, v, pos), c.run(q1, k1, v1, pos1)]

    want = [t.clone() for t in work()] + [t.clone() for t in state]
    torch.cuda.synchronize()
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap), torch.cuda.graph(graph, stream=cap):
        outs = work()
    torch.cuda.current_stream().wait_stream(cap)
    torch.cuda.synchronize()
    for rep in range(3):
        for t, t0 in zip(state, start):
            t.copy_(t0)
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs + state, want):
            assert torch.equal(x, y), f"replay {rep} differs from eager"


def test_two_streams_at_once():
    """Calls on two streams, each with its own state and workspace, give what
    they give alone; a stream can also be named."""
    require_gpu()
    announce("two streams: scan and attention side by side")
    gen = torch.Generator().manual_seed(5)
    B, T = 1, 500
    s, c = Scan(gen, B), Attention(gen, B, T)
    x, dt = rnd(gen, B, T, sum(s.widths)).to(BF).to(DEV), rnd(gen, B, T, s.H).to(DEV)
    q, k, v = (rnd(gen, B, T, h, 64).to(BF).to(DEV) for h in (8, 2, 2))
    pos = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = s.prompt(x, dt).clone(), c.run(q, k, v, pos).clone()
    S = s.S.clone()
    for rep in range(3):
        s.S.zero_()
        s.conv.zero_()
        torch.cuda.synchronize()
        sides = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(sides[0]):
            y = s.prompt(x, dt)
        with torch.cuda.stream(sides[1]):
            o = c.run(q, k, v, pos)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(o, want[1]) and torch.equal(s.S, S)
    side = torch.cuda.Stream()
    out = torch.empty(1, sum(s.widths), dtype=BF, device=DEV)
    ref_out = torch.empty_like(out)
    st = s.conv.clone()
    gdr.gdr_conv_step(x[:, 0], s.w, s.bias, s.conv, ref_out)
    torch.cuda.synchronize()
    gdr.gdr_conv_step(x[:, 0], s.w, s.bias, st, out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref_out) and torch.equal(st, s.conv)
