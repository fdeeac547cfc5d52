"""ctypes binding of libgdr.so (include/gdr.h) for torch device tensors.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  torch supplies device memory and the current
stream.  The binding checks that each tensor matches the sizes it is passed
with (device, dtype, contiguity, element count) before handing raw pointers
over, so that a wrong tensor is a Python error rather than an out-of-bounds
access.  If the library has not been built, every call raises: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import functools
from pathlib import Path

import torch

GDR_F32, GDR_BF16 = 0, 1
GDR_GATE_CHANNEL, GDR_GATE_SCALAR, GDR_GATE_SCALAR_FUSED = 0, 1, 2
GDR_OK = 0

LIB_PATH = Path(__file__).resolve().parent / "libgdr.so"
EXPORTED = ("gdr_decode_step", "gdr_prefill_workspace_size", "gdr_prefill_chunked",
            "gdr_prefill_chunked_noalloc", "gdr_conv_step", "gdr_conv_prefill", "gdr_ssm_step",
            "gdr_ssm_workspace_size", "gdr_ssm_prefill", "gdr_kv_append",
            "gdr_attn_workspace_size", "gdr_attn_cached", "gdr_strerror")
NOALLOC_SCRATCH_BYTES = 128 << 20   # GDR_NOALLOC_SCRATCH_BYTES


class GdrError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {gdr_strerror(status)} (status {status})")
        self.status = status


class gdr_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H_qk", "H_v", "dk", "dv", "chunk")]


class gdr_conv_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "W", "c0", "c1", "c2")]


class gdr_ssm_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "G", "H", "N", "P")]


class gdr_kv_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32)
                for n in ("B", "T", "H_q", "H_kv", "D", "page", "n_pages", "max_pages")]


def _sized(struct):
    """Dimension structs by their sizes: a serving loop repeats a few.  ctypes would
    wrap a size past 32 bits without a word."""
    @functools.lru_cache(maxsize=256)
    def make(*sizes):
        for (name, _), n in zip(struct._fields_, sizes):
            if not -2 ** 31 <= n < 2 ** 31:
                raise ValueError(f"{name} = {n} does not fit 32 bits")
        return struct(*sizes)
    return make


_dims, _conv_dims, _ssm_dims, _kv_dims = map(
    _sized, (gdr_dims, gdr_conv_dims, gdr_ssm_dims, gdr_kv_dims))

_lib = None


def load_library(path: Path | str | None = None):
    """Load libgdr.so (once) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path else LIB_PATH
    if not p.exists():
        raise RuntimeError(f"{p} is missing: build it with `python -m gated_delta_rule_40_amd.build`")
    lib = ctypes.CDLL(str(p))
    vp, fp, i32 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
    dims_p = ctypes.POINTER(gdr_dims)
    lib.gdr_decode_step.argtypes = [dims_p, i32, i32, vp, fp, fp, fp, fp, fp, vp,
                                    ctypes.c_float, i32, vp]
    lib.gdr_decode_step.restype = i32
    lib.gdr_prefill_workspace_size.argtypes = [dims_p, i32, i32]
    lib.gdr_prefill_workspace_size.restype = ctypes.c_size_t
    lib.gdr_prefill_chunked.argtypes = [dims_p, i32, i32, vp, vp, vp, fp, fp, fp, fp, fp, fp, vp,
                                        ctypes.c_float, i32, vp, ctypes.c_size_t, vp]
    lib.gdr_prefill_chunked.restype = i32
    lib.gdr_prefill_chunked_noalloc.argtypes = [dims_p, i32, i32, vp, vp, vp, fp, fp, fp, fp, fp,
                                                fp, vp, ctypes.c_float, i32, vp]
    lib.gdr_prefill_chunked_noalloc.restype = i32
    size, i64, f32 = ctypes.c_size_t, ctypes.c_int64, ctypes.c_float
    conv_p, ssm_p, kv_p = (ctypes.POINTER(t) for t in (gdr_conv_dims, gdr_ssm_dims, gdr_kv_dims))
    lib.gdr_conv_step.argtypes = [conv_p, i32, i32, vp, i64, vp, vp, vp, vp, vp]
    lib.gdr_conv_prefill.argtypes = [conv_p, i32, i32, vp, i64] + [vp] * 9
    lib.gdr_ssm_step.argtypes = [ssm_p, i32] + [vp] * 8
    lib.gdr_ssm_workspace_size.argtypes = [ssm_p, i32]
    lib.gdr_ssm_prefill.argtypes = [ssm_p, i32] + [vp] * 12 + [size, vp]
    lib.gdr_kv_append.argtypes = [kv_p, i32] + [vp] * 10
    lib.gdr_attn_workspace_size.argtypes = [kv_p, i32]
    lib.gdr_attn_cached.argtypes = [kv_p, i32] + [vp] * 9 + [f32, vp, size, vp]
    for name in ("gdr_conv_step", "gdr_conv_prefill", "gdr_ssm_step", "gdr_ssm_prefill",
                 "gdr_kv_append", "gdr_attn_cached"):
        getattr(lib, name).restype = i32
    lib.gdr_ssm_workspace_size.restype = lib.gdr_attn_workspace_size.restype = size
    lib.gdr_strerror.argtypes = [i32]
    lib.gdr_strerror.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def gdr_strerror(status: int) -> str:
    return load_library().gdr_strerror(int(status)).decode()


def _io_code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return GDR_F32
    if dtype == torch.bfloat16:
        return GDR_BF16
    raise ValueError(f"io dtype must be float32 or bfloat16, got {dtype}")


def _check(t, name, numel, dtype, device, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def gdr_decode_step(qkv, gate_in, beta_logit, state, o, *, H_qk, H_v, dk, dv, gate,
                    A_log=None, dt_bias=None, scale=1.0, l2norm_qk=True, stream=None):
    """One fused decode token.  qkv [B, 2*H_qk*dk + H_v*dv] (float32 or bfloat16),
    gate_in [B,H_v,dk] or [B,H_v], beta_logit [B,H_v], state [B,H_v,dk,dv] fp32
    (updated in place), o [B,H_v,dv] in qkv's dtype."""
    lib = load_library()
    B = qkv.shape[0]
    dev = qkv.device
    io = _io_code(qkv.dtype)
    f32 = torch.float32
    width = 2 * H_qk * dk + H_v * dv
    gate_n = B * H_v * dk if gate == GDR_GATE_CHANNEL else B * H_v
    fused = gate == GDR_GATE_SCALAR_FUSED
    args = (
        _check(qkv, "qkv", B * width, qkv.dtype, dev),
        _check(gate_in, "gate_in", gate_n, f32, dev),
        _check(A_log, "A_log", H_v, f32, dev, required=fused),
        _check(dt_bias, "dt_bias", H_v, f32, dev, required=fused),
        _check(beta_logit, "beta_logit", B * H_v, f32, dev),
        _check(state, "state", B * H_v * dk * dv, f32, dev),
        _check(o, "o", B * H_v * dv, qkv.dtype, dev),
    )
    dims = _dims(B, 1, H_qk, H_v, dk, dv, 0)
    rc = lib.gdr_decode_step(ctypes.byref(dims), io, int(gate), args[0], args[1], args[2],
                             args[3], args[4], args[5], args[6], float(scale), int(bool(l2norm_qk)),
                             _stream(dev, stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_decode_step")


def gdr_prefill_workspace_size(B, T, H_qk, H_v, dk, dv, chunk, io_dtype, gate) -> int:
    dims = _dims(B, T, H_qk, H_v, dk, dv, chunk)
    return int(load_library().gdr_prefill_workspace_size(ctypes.byref(dims), _io_code(io_dtype),
                                                         int(gate)))


def _prefill_args(q, k, v, gate_in, beta_logit, state_in, state_out, o, H_qk, H_v, dk, dv,
                  gate, A_log, dt_bias):
    B, T = q.shape[0], q.shape[1]
    dev = q.device
    f32 = torch.float32
    gate_n = B * T * H_v * dk if gate == GDR_GATE_CHANNEL else B * T * H_v
    fused = gate == GDR_GATE_SCALAR_FUSED
    st = B * H_v * dk * dv
    return (
        _check(q, "q", B * T * H_qk * dk, q.dtype, dev),
        _check(k, "k", B * T * H_qk * dk, q.dtype, dev),
        _check(v, "v", B * T * H_v * dv, q.dtype, dev),
        _check(gate_in, "gate_in", gate_n, f32, dev),
        _check(A_log, "A_log", H_v, f32, dev, required=fused),
        _check(dt_bias, "dt_bias", H_v, f32, dev, required=fused),
        _check(beta_logit, "beta_logit", B * T * H_v, f32, dev),
        _check(state_in, "state_in", st, f32, dev, required=False),
        _check(state_out, "state_out", st, f32, dev),
        _check(o, "o", B * T * H_v * dv, q.dtype, dev),
    )


def gdr_prefill_chunked(q, k, v, gate_in, beta_logit, state_in, state_out, o, workspace, *,
                        H_qk, H_v, dk, dv, chunk, gate, A_log=None, dt_bias=None, scale=1.0,
                        l2norm_qk=True, stream=None):
    """Chunked prefill.  q, k [B,T,H_qk,dk], v [B,T,H_v,dv] (float32 or bfloat16),
    gate_in [B,T,H_v,dk] or [B,T,H_v], beta_logit [B,T,H_v], state_in (or None)
    and state_out [B,H_v,dk,dv] fp32, o [B,T,H_v,dv], workspace a uint8 tensor
    of at least gdr_prefill_workspace_size() bytes."""
    lib = load_library()
    dev = q.device
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the same device")
        ws_ptr = ctypes.c_void_p(workspace.data_ptr())
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        ws_ptr, ws_bytes = None, 0
    args = _prefill_args(q, k, v, gate_in, beta_logit, state_in, state_out, o, H_qk, H_v, dk, dv,
                         gate, A_log, dt_bias)
    dims = _dims(q.shape[0], q.shape[1], H_qk, H_v, dk, dv, chunk)
    rc = lib.gdr_prefill_chunked(ctypes.byref(dims), _io_code(q.dtype), int(gate), *args,
                                 float(scale), int(bool(l2norm_qk)), ws_ptr,
                                 ctypes.c_size_t(ws_bytes), _stream(dev, stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_prefill_chunked")


def gdr_prefill_chunked_noalloc(q, k, v, gate_in, beta_logit, state_in, state_out, o, *,
                                H_qk, H_v, dk, dv, chunk, gate, A_log=None, dt_bias=None,
                                scale=1.0, l2norm_qk=True, stream=None):
    """gdr_prefill_chunked with the library's own device scratch as workspace
    (nothing is allocated; at most NOALLOC_SCRATCH_BYTES of workspace; calls
    that overlap on one device race on the scratch)."""
    lib = load_library()
    args = _prefill_args(q, k, v, gate_in, beta_logit, state_in, state_out, o, H_qk, H_v, dk, dv,
                         gate, A_log, dt_bias)
    dims = _dims(q.shape[0], q.shape[1], H_qk, H_v, dk, dv, chunk)
    rc = lib.gdr_prefill_chunked_noalloc(ctypes.byref(dims), _io_code(q.dtype), int(gate), *args,
                                         float(scale), int(bool(l2norm_qk)),
                                         _stream(q.device, stream))
    if rc != GDR_OK:
        raise GdrError(rc, "gdr_prefill_chunked_noalloc")


# ---------------------------------------------------------------------------
# The layers beside the gated delta rule.  Sizes are read from the tensors; the
# launch goes to the tensors' device whatever the current one is.
# ---------------------------------------------------------------------------
_F8 = (torch.float8_e4m3fn, torch.uint8)
_F32, _I32 = torch.float32, torch.int32
_IO = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16}


def _refuse(t, name, shape, dtype, device):
    """Raises with what is wrong with a tensor of a call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


# _ptr(t, name, shape, dtype, device): the address of a dense tensor of exactly
# this shape, dtype and device (native, through _refuse for all others); _opt:
# the same, None for None.
try:
    from . import _marshal
except ImportError as _why:
    _unloaded = _why  # missing, or built for another torch or Python

    def _ptr(*_):
        raise RuntimeError(f"_marshal.so cannot be loaded ({_unloaded}): build it with "
                           "`python -m gated_delta_rule_40_amd.build`") from _unloaded
    _opt = _ptr
else:
    _marshal.on_refusal(_refuse)
    _ptr, _opt = _marshal.ptr, _marshal.opt


def _lead(t, name, dims):
    """Shape, dtype code and device of the tensor that sets the sizes of a call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape, device = t.shape, t.device
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {len(shape)}")
    if device.type != "cuda":
        raise ValueError(f"{name} is on {device}, expected a GPU")
    io = _IO.get(t.dtype)
    return shape, _io_code(t.dtype) if io is None else io, device

# The current stream's handle as an integer, and the current device: torch's own
# accessors where there are any (0.1 us), else through a Stream object (2 us) and
# torch.cuda (0.3 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(name, dev, stream, *args):
    """Calls an entry point with the stream as its last argument, on `dev`."""
    fn = getattr(_lib or load_library(), name)
    index, here = dev.index, _device()
    if index == here:
        rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != GDR_OK:
        raise GdrError(rc, name)


def _taps(weight):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [C,W]")
    return weight.shape[1]


def gdr_conv_step(x, weight, bias, state, y, *, silu=True, stream=None):
    """One token of the short causal convolution.  x [B,C] (float32 or bfloat16;
    its rows may lie apart, as in a slice of a wider row), weight [C,W] fp32,
    bias [C] fp32 or None, state [B,W-1,C] in x's dtype (oldest input first,
    updated in place), y [B,C]."""
    (B, C), io, dev = _lead(x, "x", 2)
    W = _taps(weight)
    row = x.stride(0) if B > 1 else C
    if x.stride(1) != 1 and C > 1:
        raise ValueError("x's channels must be contiguous")
    _launch("gdr_conv_step", dev, stream, _conv_dims(B, 1, W, C, 0, 0), io, int(bool(silu)),
            x.data_ptr(), row, _ptr(weight, "weight", (C, W), _F32, dev),
            _opt(bias, "bias", (C,), _F32, dev), _ptr(state, "state", (B, W - 1, C), x.dtype, dev),
            _ptr(y, "y", (B, C), x.dtype, dev))


def gdr_conv_prefill(x, weight, bias, state_in, state_out, outs, *, silu=True, lens=None,
                     stream=None):
    """The short causal convolution over T tokens.  x [B,T,C] (tokens may lie
    apart, evenly over the whole batch), weight [C,W], bias [C] or None,
    state_in (or None) and state_out [B,W-1,C], outs one to three tensors
    [B,T,c] whose widths add up to C, lens [B] int32 or None."""
    (B, T, C), io, dev = _lead(x, "x", 3)
    W = _taps(weight)
    if x.is_contiguous():
        row = C
    else:
        row = x.stride(1) if T > 1 else x.stride(0) if B > 1 else C
        if (x.stride(2) != 1 and C > 1) or (T > 1 and B > 1 and x.stride(0) != T * row):
            raise ValueError("x must be rows of contiguous channels, evenly apart")
    if not 1 <= len(outs) <= 3:
        raise ValueError(f"one to three outputs, got {len(outs)}")
    c = [o.shape[-1] for o in outs]
    if sum(c) != C or 0 in c:
        raise ValueError(f"outputs of widths {c} do not split {C} channels")
    ys = [_ptr(o, f"outs[{i}]", (B, T, c[i]), x.dtype, dev) for i, o in enumerate(outs)]
    c += [0] * (3 - len(c))
    ys += [None] * (3 - len(ys))
    st = (B, W - 1, C)
    _launch("gdr_conv_prefill", dev, stream, _conv_dims(B, T, W, *c), io, int(bool(silu)),
            x.data_ptr(), row, _ptr(weight, "weight", (C, W), _F32, dev),
            _opt(bias, "bias", (C,), _F32, dev), _opt(lens, "lens", (B,), _I32, dev),
            _opt(state_in, "state_in", st, x.dtype, dev),
            _ptr(state_out, "state_out", st, x.dtype, dev), *ys)


def gdr_ssm_step(xbc, dt, A_log, dt_bias, D, state, y, *, G, H, N, P, stream=None):
    """One token of the selective state space scan.  xbc [B, H*P + 2*G*N]
    (float32 or bfloat16), dt [B,H] fp32, A_log [H], dt_bias and D [H] or None,
    state [B,H,N,P] fp32 (updated in place), y [B,H,P] in xbc's dtype."""
    (B, width), io, dev = _lead(xbc, "xbc", 2)
    _launch("gdr_ssm_step", dev, stream, _ssm_dims(B, 1, G, H, N, P), io,
            _ptr(xbc, "xbc", (B, H * P + 2 * G * N), xbc.dtype, dev),
            _ptr(dt, "dt", (B, H), _F32, dev), _ptr(A_log, "A_log", (H,), _F32, dev),
            _opt(dt_bias, "dt_bias", (H,), _F32, dev), _opt(D, "D", (H,), _F32, dev),
            _ptr(state, "state", (B, H, N, P), _F32, dev), _ptr(y, "y", (B, H, P), xbc.dtype, dev))


def gdr_ssm_workspace_size(B, T, G, H, N, P, io_dtype) -> int:
    return int(load_library().gdr_ssm_workspace_size(_ssm_dims(B, T, G, H, N, P),
                                                     _io_code(io_dtype)))


def _space(workspace, dev):
    if workspace is None:
        return None, 0
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gdr_ssm_prefill(x, b, c, dt, A_log, dt_bias, D, state_in, state_out, y, workspace, *,
                    G, H, N, P, lens=None, stream=None):
    """The selective state space scan over T tokens.  x [B,T,H,P], b and c
    [B,T,G,N] (float32 or bfloat16; dense, the last two dimensions may come as
    one), dt [B,T,H] fp32, A_log [H], dt_bias and D [H] or None, state_in (or
    None) and state_out [B,H,N,P] fp32, y like x, workspace a uint8 tensor of
    at least gdr_ssm_workspace_size() bytes (None if that is 0), lens [B] int32
    or None."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError("x must be a tensor [B,T,H,P] or [B,T,H*P]")
    shape, io, dev = _lead(x, "x", x.dim())
    B, T = shape[:2]

    def rows(t, name, heads, width):
        flat = isinstance(t, torch.Tensor) and t.dim() == 3
        return _ptr(t, name, (B, T, heads * width) if flat else (B, T, heads, width), x.dtype, dev)

    st = (B, H, N, P)
    ws, ws_bytes = _space(workspace, dev)
    _launch("gdr_ssm_prefill", dev, stream, _ssm_dims(B, T, G, H, N, P), io,
            rows(x, "x", H, P), rows(b, "b", G, N), rows(c, "c", G, N),
            _ptr(dt, "dt", (B, T, H), _F32, dev), _ptr(A_log, "A_log", (H,), _F32, dev),
            _opt(dt_bias, "dt_bias", (H,), _F32, dev), _opt(D, "D", (H,), _F32, dev),
            _opt(lens, "lens", (B,), _I32, dev), _opt(state_in, "state_in", st, _F32, dev),
            _ptr(state_out, "state_out", st, _F32, dev), rows(y, "y", H, P), ws, ws_bytes)


def _pool_heads(k_cache):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a tensor [n_pages,H_kv,page,D]")
    return k_cache.shape[1]


def _cache_args(k_cache, v_cache, k_scale, v_scale, block_table, pos, lens, B, H_kv, D, dev):
    """Pool sizes and addresses of the cache's tensors."""
    _pool_heads(k_cache)
    if k_cache.dtype not in _F8:
        raise ValueError(f"k_cache has dtype {k_cache.dtype}, expected float8_e4m3fn or uint8")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor [B,max_pages]")
    n_pages, page, per = k_cache.shape[0], k_cache.shape[2], block_table.shape[1]
    f8 = k_cache.dtype
    return (page, n_pages, per), (
        _ptr(k_cache, "k_cache", (n_pages, H_kv, page, D), f8, dev),
        _ptr(v_cache, "v_cache", (n_pages, H_kv, D, page), f8, dev),
        _ptr(k_scale, "k_scale", (n_pages, H_kv), _F32, dev),
        _ptr(v_scale, "v_scale", (n_pages, H_kv), _F32, dev),
        _ptr(block_table, "block_table", (B, per), _I32, dev), _ptr(pos, "pos", (B,), _I32, dev),
        _opt(lens, "lens", (B,), _I32, dev))


def gdr_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, pos, *, lens=None,
                  stream=None):
    """Writes new tokens' keys and values, k and v [B,T,H_kv,D] (float32 or
    bfloat16), into their pages: k_cache [n_pages,H_kv,page,D] and v_cache
    [n_pages,H_kv,D,page] (float8_e4m3fn or uint8), k_scale and v_scale
    [n_pages,H_kv] fp32, block_table [B,max_pages], pos and lens [B] int32."""
    (B, T, H_kv, D), io, dev = _lead(k, "k", 4)
    sizes, (kc, vc, ks, vs, bt, ps, ln) = _cache_args(k_cache, v_cache, k_scale, v_scale,
                                                      block_table, pos, lens, B, H_kv, D, dev)
    _launch("gdr_kv_append", dev, stream, _kv_dims(B, T, 0, H_kv, D, *sizes), io,
            _ptr(k, "k", (B, T, H_kv, D), k.dtype, dev), _ptr(v, "v", (B, T, H_kv, D), k.dtype, dev),
            bt, ps, ln, kc, vc, ks, vs)


def gdr_attn_workspace_size(B, T, H_q, H_kv, D, page, max_pages, io_dtype) -> int:
    return int(load_library().gdr_attn_workspace_size(
        _kv_dims(B, T, H_q, H_kv, D, page, 0, max_pages), _io_code(io_dtype)))


def gdr_attn_cached(q, k_cache, v_cache, k_scale, v_scale, block_table, pos, o, workspace=None, *,
                    scale, lens=None, stream=None):
    """Attention of T new tokens per row over the cache.  q and o [B,T,H_q,D]
    (float32 or bfloat16); the cache, block_table, pos and lens as in
    gdr_kv_append, with the new tokens already written; workspace a uint8
    tensor of at least gdr_attn_workspace_size() bytes (None if that is 0)."""
    (B, T, H_q, D), io, dev = _lead(q, "q", 4)
    H_kv = _pool_heads(k_cache)
    sizes, (kc, vc, ks, vs, bt, ps, ln) = _cache_args(k_cache, v_cache, k_scale, v_scale,
                                                      block_table, pos, lens, B, H_kv, D, dev)
    ws, ws_bytes = _space(workspace, dev)
    _launch("gdr_attn_cached", dev, stream, _kv_dims(B, T, H_q, H_kv, D, *sizes), io,
            _ptr(q, "q", (B, T, H_q, D), q.dtype, dev), kc, vc, ks, vs, bt, ps, ln,
            _ptr(o, "o", (B, T, H_q, D), q.dtype, dev), float(scale), ws, ws_bytes)
