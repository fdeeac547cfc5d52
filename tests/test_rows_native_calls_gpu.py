"""Plain calls of the norms, the 8-bit product and the rotary positions do go through the
native path, and it takes the current stream: captured into a graph, and on a stream that
is made the current one."""

import pytest
import torch

import gated_delta_rule_40_amd as gdr
from gated_delta_rule_40_amd import binding
from tests.gpu_util import DEV, announce, require_gpu

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _rand(*shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DEV, dtype)


class Prepared:
    """A call with everything that it takes in place: `run` makes it, `reset` brings inputs
    and outputs back to where they were, `outs` are what it writes."""

    def __init__(self, run, inputs, outs):
        self.run, self.inputs, self.outs = run, inputs, outs
        self.kept = [t.clone() for t in inputs + outs]

    def reset(self):
        for t, k in zip(self.inputs + self.outs, self.kept):
            t.copy_(k)

    def results(self):
        return [t.view(torch.uint8).clone() for t in self.outs]


def _norm(dtype, *, two=False, gate=None, apart=0, residual=None, codes_type=torch.uint8):
    R, H, D = 5, 4, 64
    x = _rand(R, H * D + apart, dtype=dtype)[:, :H * D]
    w = _rand(H, D, dtype=torch.float32, seed=1) if two else None
    g = _rand(R, H * D + apart, dtype=dtype, seed=2)[:, :H * D] if gate else None
    r = [] if residual is None else [_rand(R, H * D, dtype=residual, seed=3)]
    y = torch.zeros(R, H * D, dtype=dtype, device=DEV)
    c, s = torch.zeros(R, H * D, device=DEV).to(codes_type), torch.zeros(R, 2, device=DEV)

    def run():
        gdr.gdr_rms_norm(x, w, y, c, s, residual=r[0] if r else None, gate=g,
                         gate_first=gate == "first", heads=H, eps=1e-5)
    return Prepared(run, [x], [y, c, s] + r)


def _quant(dtype, K):
    x = _rand(7, K, dtype=dtype)
    c, s = torch.zeros(7, K, device=DEV).to(F8), torch.zeros(7, -(-K // 128), device=DEV)
    return Prepared(lambda: gdr.gdr_quant_rows(x, c, s), [x], [c, s])


def _matmul(dtype, bias, M=9):
    N, K = 130, 208
    x, w = (_rand(n, K, dtype=torch.float32, seed=n).to(F8) for n in (M, N))
    sx, sw = (_rand(n, 2, dtype=torch.float32, seed=n).abs() for n in (M, 2))
    b = _rand(N, dtype=torch.float32, seed=6) if bias else None
    y = torch.zeros(M, N, dtype=dtype, device=DEV)
    return Prepared(lambda: gdr.gdr_matmul_fp8(x, sx, w, sw, y, bias=b), [x], [y])


def _rope(dtype, v, apart, interleaved, ragged):
    B, T, Hq, Hkv, D = 2, 3, 4, 2, 64
    C = (Hq + (1 + v) * Hkv) * D
    x = _rand(B, T, C + apart, dtype=dtype)[:, :, :C]
    freq, m = gdr.gdr_rope_freqs(32, 10000.0)
    freq = freq.to(DEV)
    outs = [torch.zeros(B, T, h, D, dtype=dtype, device=DEV) for h in (Hq, Hkv, Hkv)[:2 + v]]
    pos, lens = (torch.tensor(n, dtype=torch.int32, device=DEV) for n in ([0, 17], [3, 1]))

    def run():
        gdr.gdr_rope(x, freq, pos, *outs, interleaved=interleaved, magnitude=m,
                     lens=lens if ragged else None)
    return Prepared(run, [x], outs)


CALLS = {
    "norm": lambda t: _norm(t, codes_type=F8),
    "norm_weight": lambda t: _norm(t, two=True, apart=32),
    "norm_gate": lambda t: _norm(t, two=True, gate="after", apart=32),
    "norm_gate_first": lambda t: _norm(t, gate="first"),
    "norm_sum": lambda t: _norm(t, two=True, residual=torch.float32),
    "norm_sum_16": lambda t: _norm(t, residual=torch.bfloat16),
    "quant": lambda t: _quant(t, 256),
    "quant_odd": lambda t: _quant(t, 131),
    "matmul": lambda t: _matmul(t, False),
    "matmul_bias": lambda t: _matmul(t, True),
    "matmul_tiles": lambda t: _matmul(t, True, M=700),
    "rope": lambda t: _rope(t, True, 0, False, False),
    "rope_apart": lambda t: _rope(t, True, 64, True, True),
    "rope_no_v": lambda t: _rope(t, False, 64, False, True),
}
NATIVE = {"norm": "_norm_call", "quant": "_quant_call", "matmul": "_matmul_call",
          "rope": "_rope_call"}
DTYPES = dict(argnames="dtype", argvalues=[torch.float32, torch.bfloat16], ids=["f32", "bf16"])


def eager(call):
    call.reset()
    call.run()
    torch.cuda.synchronize()
    want = call.results()
    assert all(bool(w.any()) for w in want)
    return want


@pytest.mark.parametrize(**DTYPES)
@pytest.mark.parametrize("name", CALLS)
def test_plain_calls_are_native(name, dtype, monkeypatch):
    require_gpu()
    announce(f"native call {name} {dtype}")
    call, seen = CALLS[name](dtype), []
    attribute = NATIVE[name.split("_")[0]]
    native = getattr(binding, attribute)

    def spy(*args):
        seen.append(native(*args))
        return seen[-1]

    monkeypatch.setattr(binding, attribute, spy)
    call.run()
    torch.cuda.synchronize()
    assert seen == [0]                  # None: left to the Python path


@pytest.mark.parametrize(**DTYPES)
@pytest.mark.parametrize("name", CALLS)
def test_native_calls_in_a_graph(name, dtype):
    require_gpu()
    announce(f"native call {name} {dtype} captured")
    call = CALLS[name](dtype)
    want = eager(call)
    call.reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    torch.cuda.synchronize()
    assert all(torch.equal(t, k) for t, k in zip(call.outs, call.kept[len(call.inputs):]))
    for _ in range(3):
        call.reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(call.results(), want))
        torch.randn(1000, device=DEV).sum().item()


@pytest.mark.parametrize(**DTYPES)
@pytest.mark.parametrize("name", CALLS)
def test_native_calls_on_a_stream_made_current(name, dtype):
    """Its inputs come late on that stream: a call on any other would read zeros."""
    require_gpu()
    announce(f"native call {name} {dtype} on a stream made current")
    call = CALLS[name](dtype)
    want = eager(call)
    call.reset()
    for t in call.inputs:
        t.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)    # cycles: a millisecond or so
        for t, k in zip(call.inputs, call.kept):
            t.copy_(k)
        call.run()
        for t in call.inputs:
            t.zero_()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(call.results(), want))
