"""Norms, 8-bit products and rotary positions together with the mixers between them,
as a layer calls them: a prompt and single tokens, captured in a graph and replayed,
and on other streams.  Each stage is held to its 64-bit form on the inputs that it got."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_40_amd as gdr
import oracle
from tests import layer_ref, rows_ref as ref
from tests.gpu_util import DEV, announce, require_gpu

pytestmark = pytest.mark.gpu

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
HID = 384


def quantised(gen, N, K):
    """A weight [N,K] as codes with a scale per 128 x 128."""
    w = torch.randn(N, K, generator=gen) / math.sqrt(K)
    nb, kb = -(-N // 128), -(-K // 128)
    top = torch.zeros(nb, kb)
    for i in range(nb):
        for j in range(kb):
            top[i, j] = w[i * 128: i * 128 + 128, j * 128: j * 128 + 128].abs().max()
    sw = top / 448
    full = sw.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return (w / full).to(F8).to(DEV), sw.to(DEV)


def rows8(R, K):
    return torch.zeros(R, K, device=DEV).to(F8), torch.zeros(R, -(-K // 128), device=DEV)


def check_norm(x, weight, eps, codes, scales, residual=None, after=None, gate=None, heads=1):
    """codes of a norm; `after`: what the residual became."""
    want, stored, units = ref.norm(x.cpu(), weight.cpu(), eps, residual, gate, False, heads)
    ref.check_codes(codes.cpu(), scales.cpu(), want, units)
    if residual is not None:
        bound = layer_ref.HALF[after.dtype] * stored.abs() + ref.U * stored.abs() + 1e-37
        assert layer_ref.worst(after.cpu(), stored, bound) <= 1


def check_product(codes, scales, w, sw, y):
    want, mag = ref.matmul(codes.cpu().double(), scales.cpu(), w.cpu().double(), sw.cpu())
    assert layer_ref.worst(y.cpu(), want, ref.matmul_bound(want, mag, y.dtype, w.shape[1])) <= 1


class DeltaLayer:
    """norm -> product -> convolution -> gated delta rule -> gated norm -> product."""
    Hq, Hv, dk, dv, W = 2, 4, 64, 64, 4

    def __init__(self, gen, B):
        self.B, self.C, self.V = B, (2 * self.Hq + self.Hv) * 64, self.Hv * 64
        self.norm = (1 + 0.2 * torch.randn(HID, generator=gen)).to(DEV)
        self.gated = (1 + 0.2 * torch.randn(self.Hv, self.dv, generator=gen)).to(DEV)
        self.w_in, self.s_in = quantised(gen, self.C + self.V, HID)
        self.w_out, self.s_out = quantised(gen, HID, self.V)
        self.taps = (torch.randn(self.C, self.W, generator=gen) * 0.6).to(DEV)
        self.conv = torch.zeros(B, self.W - 1, self.C, dtype=BF, device=DEV)
        self.S = torch.zeros(B, self.Hv, self.dk, self.dv, device=DEV)
        self.kw = dict(H_qk=self.Hq, H_v=self.Hv, dk=self.dk, dv=self.dv,
                       gate=gdr.GDR_GATE_SCALAR, scale=1 / math.sqrt(self.dk))
        self.token_rows = None

    def rows(self, R):
        return dict(c0=rows8(R, HID), c1=rows8(R, self.V),
                    packed=torch.empty(R, self.C + self.V, dtype=BF, device=DEV),
                    out=torch.empty(R, HID, dtype=BF, device=DEV))

    def enter(self, x, residual, t):
        gdr.gdr_rms_norm(x, self.norm, None, *t["c0"], residual=residual)
        gdr.gdr_matmul_fp8(*t["c0"], self.w_in, self.s_in, t["packed"])

    def leave(self, o, t):
        z = t["packed"][:, self.C:]                       # rows that lie apart
        gdr.gdr_rms_norm(o.view(-1, self.V), self.gated, None, *t["c1"], gate=z)
        gdr.gdr_matmul_fp8(*t["c1"], self.w_out, self.s_out, t["out"])
        return t["out"]

    def prompt(self, x, residual, g, beta):
        B, T = self.B, x.shape[0] // self.B
        t = self.rows(B * T)
        self.enter(x, residual, t)
        packed = t["packed"].view(B, T, -1)[:, :, : self.C]
        t["qkv"] = [torch.empty(B, T, c, dtype=BF, device=DEV) for c in
                    (self.Hq * 64, self.Hq * 64, self.Hv * 64)]
        gdr.gdr_conv_prefill(packed, self.taps, None, self.conv, self.conv, t["qkv"])
        t["o"] = torch.empty(B, T, self.Hv, self.dv, dtype=BF, device=DEV)
        ws = torch.empty(gdr.gdr_prefill_workspace_size(B, T, self.Hq, self.Hv, 64, 64, 32, BF,
                                                        gdr.GDR_GATE_SCALAR),
                         dtype=torch.uint8, device=DEV)
        gdr.gdr_prefill_chunked(*t["qkv"], g, beta, self.S, self.S, t["o"], ws, chunk=32, **self.kw)
        self.leave(t["o"], t)
        return t

    def token(self, x, residual, g, beta):
        if self.token_rows is None:
            self.token_rows = self.rows(self.B)
            self.token_rows["qkv"] = torch.empty(self.B, self.C, dtype=BF, device=DEV)
            self.token_rows["o"] = torch.empty(self.B, self.Hv, self.dv, dtype=BF, device=DEV)
        t = self.token_rows
        self.enter(x, residual, t)
        gdr.gdr_conv_step(t["packed"][:, : self.C], self.taps, None, self.conv, t["qkv"])
        gdr.gdr_decode_step(t["qkv"], g, beta, self.S, t["o"], **self.kw)
        self.leave(t["o"], t)
        return t


def delta_inputs(gen, B, T):
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return (r(B, T, HID).to(BF), (r(B, T, HID) * 2).to(BF), -r(B, T, 4).abs() * 0.2, r(B, T, 4))


def test_delta_layer_of_a_prompt_and_of_tokens():
    require_gpu()
    announce("chain norm -> product -> conv -> delta rule -> gated norm -> product")
    gen = torch.Generator().manual_seed(1)
    B, T, n = 2, 40, 3
    m = DeltaLayer(gen, B)
    x, res, g, beta = delta_inputs(gen, B, T + n)
    up = lambda t: t.contiguous().to(DEV)  # noqa: E731
    os, packed = [], []
    for lo, hi in [(0, T)] + [(T + i, T + i + 1) for i in range(n)]:
        xs, rs = x[:, lo:hi].reshape(-1, HID), res[:, lo:hi].reshape(-1, HID)
        dr = up(rs)
        call = m.prompt if hi - lo > 1 else m.token
        gs, bs = (up(g[:, lo:hi]), up(beta[:, lo:hi])) if hi - lo > 1 else (up(g[:, lo]),
                                                                           up(beta[:, lo]))
        t = call(up(xs), dr, gs, bs)
        check_norm(xs, m.norm, 1e-6, *t["c0"], residual=rs, after=dr)
        check_product(*t["c0"], m.w_in, m.s_in, t["packed"])
        check_norm(t["o"].view(-1, m.V), m.gated, 1e-6, *t["c1"], gate=t["packed"][:, m.C:].cpu(),
                   heads=m.Hv)
        check_product(*t["c1"], m.w_out, m.s_out, t["out"])
        os.append(t["o"].reshape(B, hi - lo, m.Hv, m.dv).cpu())
        packed.append(t["packed"].view(B, hi - lo, -1)[:, :, : m.C].cpu())
    y, _, _ = layer_ref.conv(torch.cat(packed, 1), m.taps.cpu(), None, None)
    q, k, v = (a.reshape(B, T + n, -1, 64).numpy() for a in
               y.to(BF).double().split([m.Hq * 64, m.Hq * 64, m.Hv * 64], -1))
    o, S = oracle.sequence(q, k, v, gdr.GDR_GATE_SCALAR, g.numpy(), beta.numpy(), None,
                           scale=1 / math.sqrt(m.dk))
    assert layer_ref.rel(torch.cat(os, 1), torch.from_numpy(o)) < 2e-2
    assert layer_ref.rel(m.S.cpu(), torch.from_numpy(S)) < 2e-2


class AttentionLayer:
    """norm -> product -> rotary -> cache -> attention -> plain 8 bits -> product."""
    Hq, Hkv, D, page, per = 4, 2, 64, 16, 6

    def __init__(self, gen, B):
        self.B, self.C = B, (self.Hq + 2 * self.Hkv) * self.D
        self.norm = (1 + 0.2 * torch.randn(HID, generator=gen)).to(DEV)
        self.w_in, self.s_in = quantised(gen, self.C, HID)
        self.w_out, self.s_out = quantised(gen, HID, self.Hq * self.D)
        freq, self.magnitude = gdr.gdr_rope_freqs(32, 10000.0, kind=gdr.GDR_ROPE_INDEX, factor=4.0,
                                                  context=64.0, low=1.0, high=8.0)
        self.freq = freq.to(DEV)
        n = B * self.per
        self.table = torch.randperm(n, generator=gen).view(B, -1).to(torch.int32).to(DEV)
        z = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
        self.cache = (z(n, self.Hkv, self.page, self.D).to(F8), z(n, self.Hkv, self.D, self.page)
                      .to(F8), z(n, self.Hkv), z(n, self.Hkv), self.table)

    def run(self, x, residual, pos, T, lens=None):
        B = self.B
        t = dict(c0=rows8(B * T, HID), c1=rows8(B * T, self.Hq * self.D),
                 packed=torch.zeros(B, T, self.C, dtype=BF, device=DEV),
                 out=torch.zeros(B * T, HID, dtype=BF, device=DEV))
        for n, h in (("q", self.Hq), ("k", self.Hkv), ("v", self.Hkv), ("o", self.Hq)):
            t[n] = torch.zeros(B, T, h, self.D, dtype=BF, device=DEV)
        gdr.gdr_rms_norm(x, self.norm, None, *t["c0"], residual=residual)
        gdr.gdr_matmul_fp8(*t["c0"], self.w_in, self.s_in, t["packed"].view(B * T, self.C))
        gdr.gdr_rope(t["packed"], self.freq, pos, t["q"], t["k"], t["v"], lens=lens,
                     magnitude=self.magnitude)
        gdr.gdr_kv_append(t["k"], t["v"], *self.cache, pos, lens=lens)
        size = gdr.gdr_attn_workspace_size(B, T, self.Hq, self.Hkv, self.D, self.page, self.per, BF)
        ws = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
        gdr.gdr_attn_cached(t["q"], *self.cache, pos, t["o"], ws, scale=1 / 8, lens=lens)
        gdr.gdr_quant_rows(t["o"].view(B * T, -1), *t["c1"])
        gdr.gdr_matmul_fp8(*t["c1"], self.w_out, self.s_out, t["out"])
        return t


def test_attention_layer_of_a_padded_prompt_and_of_tokens():
    require_gpu()
    announce("chain norm -> product -> rotary -> cache -> attention -> 8 bits -> product")
    gen = torch.Generator().manual_seed(2)
    B = 3
    m = AttentionLayer(gen, B)
    pos = torch.zeros(B, dtype=torch.int32)
    for T, lens in [(37, [37, 20, 1]), (1, None), (1, None), (5, [5, 0, 3])]:
        x = torch.randn(B * T, HID, generator=gen).to(BF)
        res = (torch.randn(B * T, HID, generator=gen) * 2).to(BF)
        dr = res.to(DEV)
        gl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
        t = m.run(x.to(DEV), dr, pos.to(DEV), T, gl)
        check_norm(x, m.norm, 1e-6, *t["c0"], residual=res, after=dr)
        check_product(*t["c0"], m.w_in, m.s_in, t["packed"].view(B * T, -1))
        want, mag = ref.rope(t["packed"].cpu(), m.freq.cpu(), pos, m.Hq, m.Hkv, m.D, False,
                             m.magnitude, lens)
        got = torch.cat([t["q"], t["k"], t["v"]], 2).cpu()
        assert layer_ref.worst(got, want, ref.rope_bound(want, mag, BF) + 1e-37) <= 1
        kc, vc, ks, vs, table = (c.cpu() for c in m.cache)
        want, mag, _ = layer_ref.attention(t["q"].cpu(), kc.double(), vc.double(), ks, vs, table,
                                           pos, 1 / 8, lens)
        assert layer_ref.rel(t["o"].cpu(), want) < 2.0 ** -8
        ref.check_codes(t["c1"][0].cpu(), t["c1"][1].cpu(), t["o"].view(B * T, -1).cpu().double(),
                        torch.zeros(B * T, m.Hq * m.D, dtype=ref.F64))
        check_product(*t["c1"], m.w_out, m.s_out, t["out"])
        pos = pos + torch.tensor([T] * B if lens is None else lens, dtype=torch.int32)


def test_tokens_replayed_from_a_graph():
    """A captured token of the layer against the eager one, over several replays with
    other work and synchronisations between them."""
    require_gpu()
    announce("chain in a graph")
    B, n = 3, 6
    x, res, g, beta = (t.to(DEV) for t in delta_inputs(torch.Generator().manual_seed(3), B, n))
    eager, captured = (DeltaLayer(torch.Generator().manual_seed(4), B) for _ in range(2))
    want = []
    for i in range(n):
        r = res[:, i].contiguous()
        t = eager.token(x[:, i].contiguous(), r, g[:, i].contiguous(), beta[:, i].contiguous())
        want.append([v.clone() for v in (t["out"], r, t["c1"][0].view(torch.uint8), t["c1"][1])])
    static = [t[:, 0].contiguous() for t in (x, res, g, beta)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.token(*static)                             # a first call outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = captured.token(*static)
    captured.conv.zero_()
    captured.S.zero_()
    for i in range(n):
        for s, v in zip(static, (x, res, g, beta)):
            s.copy_(v[:, i])
        graph.replay()
        torch.cuda.synchronize()
        torch.randn(1000, device=DEV).sum().item()
        got = (t["out"], static[1], t["c1"][0].view(torch.uint8), t["c1"][1])
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b), i
    assert torch.equal(captured.S, eager.S)


def test_calls_on_other_streams_at_once():
    require_gpu()
    announce("norm, product and rope on three streams")
    gen = torch.Generator(device=DEV).manual_seed(5)
    streams = [torch.cuda.Stream() for _ in range(3)]
    freq = gdr.gdr_rope_freqs(64, 10000.0)[0].to(DEV)

    def work(i, stream):
        R = 200 + 70 * i
        x = torch.randn(R, 512, generator=gen, device=DEV).to(BF)
        w = (torch.randn(384, 512, generator=gen, device=DEV) * 40).to(F8)
        sw = torch.rand(3, 4, generator=gen, device=DEV)
        c, s = torch.empty(R, 512, device=DEV).to(F8), torch.empty(R, 4, device=DEV)
        y = torch.empty(R, 384, dtype=BF, device=DEV)
        q, k, v = (torch.empty(1, R, h, 64, dtype=BF, device=DEV) for h in (2, 2, 2))
        pos = torch.tensor([9], dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()

        def go():
            gdr.gdr_rms_norm(x, None, None, c, s, stream=stream)
            gdr.gdr_matmul_fp8(c, s, w, sw, y, stream=stream)
            gdr.gdr_rope(y[None], freq, pos, q, k, v, stream=stream)
        return go, (c, s, y, q, k, v)

    jobs = [work(i, s) for i, s in enumerate(streams)]
    for _ in range(3):
        for go, _ in jobs:
            go()
    torch.cuda.synchronize()
    together = [[t.clone() for t in outs] for _, outs in jobs]
    for (go, outs), kept in zip(jobs, together):
        for t in outs:
            t.view(torch.uint8).zero_() if t.dtype == F8 else t.zero_()
        torch.cuda.synchronize()  # the clearing is on this stream, the calls on theirs
        go()
        torch.cuda.synchronize()
        for a, b in zip(outs, kept):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
