"""The calls of the norms, the 8-bit product and the rotary positions through the native
path (the current stream of the current device) and through the Python path (a stream
that is named): the same kernels, so the same bytes; and what one refuses, the other does."""

import pytest
import torch

import gated_delta_rule_40_amd as gdr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _rand(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DEV, dtype)


def _norm(stream, dtype, *, two=False, gate=None, apart=False, residual=None):
    R, H, D = 5, 3, 64
    x = _rand(R, H * D + 32 * apart, dtype=dtype)[:, :H * D]
    w = _rand(H, D, dtype=torch.float32, seed=1) if two else None
    g = None if gate is None else _rand(R, H * D + 32 * apart, dtype=dtype, seed=2)[:, :H * D]
    r = None if residual is None else _rand(R, H * D, dtype=residual, seed=3)
    y = torch.zeros(R, H * D, dtype=dtype, device=DEV)
    codes = torch.zeros(R, H * D, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(R, -(-H * D // 128), device=DEV)
    gdr.gdr_rms_norm(x, w, y, codes, scales, residual=r, gate=g, gate_first=gate == "first",
                     heads=H, eps=1e-5, stream=stream)
    return [y, codes, scales] + ([] if r is None else [r])


def _quant(stream, dtype, K):
    x = _rand(7, K, dtype=dtype)
    codes = torch.zeros(7, K, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.zeros(7, -(-K // 128), device=DEV)
    gdr.gdr_quant_rows(x, codes, scales, stream=stream)
    return [codes.view(torch.uint8), scales]


def _matmul(stream, dtype, bias):
    M, N, K = 9, 130, 208
    x, w = (_rand(n, K, seed=n).to(torch.float8_e4m3fn) for n in (M, N))
    sx = _rand(M, 2, dtype=torch.float32, seed=4).abs()
    sw = _rand(2, 2, dtype=torch.float32, seed=5).abs()
    b = _rand(N, dtype=torch.float32, seed=6) if bias else None
    y = torch.zeros(M, N, dtype=dtype, device=DEV)
    gdr.gdr_matmul_fp8(x, sx, w, sw, y, bias=b, stream=stream)
    return [y]


def _rope(stream, dtype, v, apart, interleaved):
    B, T, H_q, H_kv, D = 2, 3, 4, 2, 64
    C = (H_q + (1 + v) * H_kv) * D
    x = _rand(B, T, C + 64 * apart, dtype=dtype)[:, :, :C]
    freq, m = gdr.gdr_rope_freqs(32, 10000.0)
    q = torch.zeros(B, T, H_q, D, dtype=dtype, device=DEV)
    k, u = (torch.zeros(B, T, H_kv, D, dtype=dtype, device=DEV) for _ in range(2))
    pos = torch.tensor([0, 17], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    gdr.gdr_rope(x, freq.to(DEV), pos, q, k, u if v else None, interleaved=interleaved,
                 magnitude=m, lens=lens, stream=stream)
    return [q, k, u]


CALLS = {
    "norm": lambda s, t: _norm(s, t),
    "norm_weight": lambda s, t: _norm(s, t, two=True, apart=True),
    "norm_gate": lambda s, t: _norm(s, t, two=True, gate="after", apart=True),
    "norm_gate_first": lambda s, t: _norm(s, t, gate="first"),
    "norm_sum": lambda s, t: _norm(s, t, two=True, residual=torch.float32),
    "norm_sum_16": lambda s, t: _norm(s, t, residual=torch.bfloat16),
    "quant": lambda s, t: _quant(s, t, 256),
    "quant_odd": lambda s, t: _quant(s, t, 131),
    "matmul": lambda s, t: _matmul(s, t, False),
    "matmul_bias": lambda s, t: _matmul(s, t, True),
    "rope": lambda s, t: _rope(s, t, True, False, False),
    "rope_apart": lambda s, t: _rope(s, t, True, True, True),
    "rope_no_v": lambda s, t: _rope(s, t, False, True, False),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", CALLS)
def test_native_and_python_paths_agree(name, dtype):
    native = CALLS[name](None, dtype)
    named = CALLS[name](torch.cuda.current_stream(), dtype)
    torch.cuda.synchronize()
    assert any(bool(t.float().abs().sum() > 0) for t in native)
    for a, b in zip(native, named):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", CALLS)
def test_native_path_takes_the_current_stream(name):
    """Captured calls land in the graph, which takes the stream of the capture."""
    want = CALLS[name](None, torch.bfloat16)
    native = getattr(gdr.binding, "_native")
    assert native is not None
    x = _rand(5, 256)
    codes = torch.zeros(5, 256, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(5, 2, device=DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        assert native.quant_rows(x, codes, scales) == 0
    torch.cuda.synchronize()
    assert not codes.any()
    for _ in range(3):
        codes.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert codes.any()
    again = CALLS[name](None, torch.bfloat16)
    for a, b in zip(want, again):
        assert torch.equal(a, b)


def test_refusals_name_the_argument():
    x = _rand(4, 256)
    y = torch.empty_like(x)
    codes = torch.empty(4, 256, dtype=torch.uint8, device=DEV)
    scales = torch.empty(4, 2, device=DEV)
    bad = [
        (lambda: gdr.gdr_rms_norm(x, None, y[:, :128]), ValueError, "y has shape"),
        (lambda: gdr.gdr_rms_norm(x, None, y.float()), ValueError, "y has dtype"),
        (lambda: gdr.gdr_rms_norm(x, None, y.cpu()), ValueError, "y is on"),
        (lambda: gdr.gdr_rms_norm(x, None, y, heads=3), ValueError, "are not 3 heads"),
        (lambda: gdr.gdr_rms_norm(x.T, None, y.T), ValueError, "channels must be contiguous"),
        (lambda: gdr.gdr_rms_norm(x, None, y, None, scales), ValueError, "scales without codes"),
        (lambda: gdr.gdr_rms_norm(x, None, y, gate=y.float()), ValueError, "gate must be like"),
        (lambda: gdr.gdr_rms_norm(x, None, x), gdr.GdrError, "gdr_rms_norm"),
        (lambda: gdr.gdr_rms_norm(x, None, y, eps=-1.0), gdr.GdrError, "gdr_rms_norm"),
        (lambda: gdr.gdr_rms_norm(x, None, y, eps="small"), Exception, None),
        (lambda: gdr.gdr_quant_rows(x.half(), codes, scales), (TypeError, ValueError), None),
        (lambda: gdr.gdr_quant_rows(x, codes, None), (TypeError, ValueError), "scales"),
        (lambda: gdr.gdr_quant_rows(x, codes, scales.cpu()), ValueError, "scales is on"),
        (lambda: gdr.gdr_matmul_fp8(codes, scales, codes, scales, y), ValueError, "shape"),
        (lambda: gdr.gdr_matmul_fp8(x, scales, codes, scales, y), ValueError, "x must be"),
    ]
    for call, kind, words in bad:
        with pytest.raises(kind, match=words):
            call()
    torch.cuda.synchronize()
