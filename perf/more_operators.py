"""What stands between the residual stream and a layer's mixer: root-mean-square
norms, products of 8-bit matrices and rotary positions.  What is measured of them,
with their plain forms.

`run` computes an operator by elementary torch operations in 32 bits (angles in
64), or, with `own` set, calls the library.  The operators:

  norm     h = x + residual (stored back), n = h / sqrt(mean h^2 + eps) over each
           of H heads of D channels, y = n w; with a gate z: y = n w silu(z)
           ("after"), or h = x silu(z) before the norm ("before").  As rows of
           the io type, or as e4m3 codes c with a scale s per row and 128
           channels, s = max(amax / 448, 2^-100), c = y / s
  quant    rows to codes and scales without a norm
  product  y[m, n] = bias[n] + sum over blocks b of 128 of
           sx[m, b] sw[n / 128, b] sum over k in b of x[m, k] w[n, k]
  rope     packed rows of q | k | v heads split into dense tensors; the first R
           channels of each head of q and k turned by position times frequency,
           in pairs (i, i + R / 2) or (2 i, 2 i + 1)

Padded batches carry a length per row; rows behind it stay as they were.
"""
import math

import torch

own = False

DEV = "cuda:0"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One token of one request enters a layer: a call's latency.
        dict(name="norm_b1", op="norm", io="bf16", R=1, H=1, D=4096, res="bf16", gate="", out="8"),
        # A prompt of 4000 tokens enters a layer.
        dict(name="norm_t4000", op="norm", io="bf16", R=4000, H=1, D=4096, res="bf16", gate="",
             out="8"),
        # The gated delta rule's output of 64 requests, head by head, on its way to the
        # output projection.
        dict(name="norm_gated_b64", op="norm", io="bf16", R=64, H=32, D=128, res="", gate="after",
             out="8"),
        # The scan's output over a prompt, in groups of heads, gated before the norm.
        dict(name="norm_gated_t4000", op="norm", io="bf16", R=4000, H=8, D=512, res="",
             gate="before", out="io"),
        # A final norm in single precision, rows that are not of whole vectors.
        dict(name="norm_f32_odd", op="norm", io="f32", R=777, H=1, D=2501, res="f32", gate="",
             out="io"),
        # The input projection of a 16 -> 32 head layer, one token: weights streamed.
        dict(name="product_b1", op="product", io="bf16", M=1, N=8192, K=4096, bias=False),
        # The same for one token of 64 requests.
        dict(name="product_b64", op="product", io="bf16", M=64, N=8192, K=4096, bias=False),
        # The same for a prompt.
        dict(name="product_t4000", op="product", io="bf16", M=4000, N=8192, K=4096, bias=False),
        # A short prompt through a projection of odd sizes, single-precision output.
        dict(name="product_ragged", op="product", io="f32", M=333, N=1003, K=2064, bias=True),
        # One token of 64 requests on its way to the cache.
        dict(name="rope_b64", op="rope", io="bf16", B=64, T=1, Hq=32, Hkv=8, D=128, R=128,
             pairs="half", pos=8192, ragged=False),
        # A prompt.
        dict(name="rope_t4000", op="rope", io="bf16", B=1, T=4000, Hq=32, Hkv=8, D=128, R=128,
             pairs="half", pos=0, ragged=False),
        # Unequal prompts far into a long context, half of each head turned.
        dict(name="rope_far", op="rope", io="bf16", B=4, T=2047, Hq=16, Hkv=2, D=128, R=64,
             pairs="interleaved", pos=1000000, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "product", "product", "product", "rope", "rope"])
    c = dict(op=op, io=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        D = rng.choice([16, 32, 64, 128, 256, 128 * _log(rng, 1, 32), 8 * _log(rng, 1, 500),
                        _log(rng, 1, 5000)])
        H = 1 if D % 128 and D not in (16, 32, 64) else rng.choice([1, 2, 7, 32])
        kind = rng.choice(["", "res", "res", "after", "before"])
        c.update(R=_log(rng, 1, min(4000, max(1, 12_000_000 // (H * D)))), H=H, D=D,
                 res=rng.choice(["bf16", "f32"]) if kind == "res" else "",
                 gate=kind if kind != "res" else "", out=rng.choice(["8", "8", "io"]))
    elif op == "quant":
        D = rng.choice([128 * _log(rng, 1, 40), 8 * _log(rng, 1, 500), _log(rng, 1, 5000)])
        c.update(R=_log(rng, 1, 3000), D=D)
    elif op == "product":
        c.update(M=rng.choice([_log(rng, 1, 64), _log(rng, 1, 4000)]), N=_log(rng, 16, 8192),
                 K=16 * _log(rng, 1, 256), bias=rng.random() < 0.3)
    else:
        D = rng.choice([64, 128, 128, 256])
        T = rng.choice([1, _log(rng, 2, 4000)])
        c.update(T=T, B=_log(rng, 1, 128) if T == 1 else rng.randint(1, 1 + 4000 // T % 6), D=D,
                 R=rng.choice([D, D, D // 2, D // 4, D - 6]), Hq=rng.choice([1, 4, 7, 16]),
                 Hkv=rng.choice([1, 2, 4]), pairs=rng.choice(["half", "interleaved"]),
                 pos=rng.choice([0, _log(rng, 1, 2000000)]), ragged=T > 1 and rng.random() < 0.5)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _blocks(t):
    """The last dimension in blocks of 128, zeros behind its end."""
    n = -(-t.shape[-1] // BLOCK)
    t = torch.nn.functional.pad(t, (0, n * BLOCK - t.shape[-1]))
    return t.view(*t.shape[:-1], n, BLOCK)


def _prepare_norm(case, gen, io):
    def rnd(*s):
        return torch.randn(*s, generator=gen, device=DEV)

    R, H, D = case["R"], case.get("H", 1), case["D"]
    # A few channels carry much more than the others, as hidden states have it.
    size = torch.exp(rnd(H * D) * 0.8)
    s = dict(x=(rnd(R, H * D) * size).to(io))
    if case["op"] == "norm":
        s["weight"] = 1 + 0.2 * rnd(H, D)
        if case["res"]:
            s["residual"] = (rnd(R, H * D) * size * 3).to(IO[case["res"]])
        if case["gate"]:
            s["gate"] = rnd(R, H * D).to(io)
    if case.get("out") == "io":
        s["y"] = torch.empty(R, H * D, dtype=io, device=DEV)
    else:
        s["codes"] = torch.empty(R, H * D, dtype=E4M3, device=DEV)
        s["scales"] = torch.empty(R, -(-H * D // BLOCK), device=DEV)
    return s


def _prepare_product(case, gen, io):
    M, N, K = (case[k] for k in "MNK")
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    x = torch.randn(M, K, generator=gen, device=DEV)
    x *= torch.exp(torch.randn(K, generator=gen, device=DEV) * 0.8)
    sx = _blocks(x).abs().amax(-1) / 448
    w = torch.randn(N, K, generator=gen, device=DEV) / math.sqrt(K)
    w *= torch.exp(torch.randn(N, 1, generator=gen, device=DEV) * 0.3)
    pad = torch.nn.functional.pad(w, (0, 0, 0, nb * BLOCK - N)).t()
    sw = _blocks(pad.contiguous()).abs().amax(-1)                       # [K, nb]
    sw = _blocks(sw.t().contiguous()).amax(-1) / 448                    # [nb, kb]

    def up(t, d):
        return t.repeat_interleave(BLOCK, d)

    s = dict(x=(x / up(sx, 1)[:, :K]).to(E4M3), sx=sx,
             w=(w / up(up(sw, 0), 1)[:N, :K]).to(E4M3), sw=sw.contiguous(),
             y=torch.empty(M, N, dtype=io, device=DEV), bias=None)
    if case["bias"]:
        s["bias"] = torch.randn(N, generator=gen, device=DEV) * 0.5
    return s


def _prepare_rope(case, gen, io):
    B, T, Hq, Hkv, D, R = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "R"))
    i = torch.arange(R // 2, dtype=torch.float64, device=DEV)
    # Contexts past half a million tokens come with stretched frequencies.
    base = 10000.0 if case["pos"] < 500000 else 5000000.0
    pos = torch.randint(case["pos"] // 2, case["pos"] + 1, (B,), generator=gen, device=DEV)
    s = dict(x=torch.randn(B, T, (Hq + 2 * Hkv) * D, generator=gen, device=DEV).to(io),
             freq=base ** (-2 * i / R), pos=pos.to(torch.int32), lens=None,
             magnitude=1.0 if case["pos"] < 500000 else 1.1386)
    if case["ragged"]:
        s["lens"] = torch.randint(T // 2, T + 1, (B,), generator=gen, device=DEV).to(torch.int32)
    for name, heads in (("q", Hq), ("k", Hkv), ("v", Hkv)):
        s[name] = torch.zeros(B, T, heads, D, dtype=io, device=DEV)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    make = {"product": _prepare_product, "rope": _prepare_rope}.get(case["op"], _prepare_norm)
    s = make(case, gen, IO[case["io"]])
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _codes(y):
    """Codes and scales of rows in 32 bits."""
    b = _blocks(y)
    scale = (b.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
    c = (b / scale[..., None]).clamp(-448, 448).flatten(-2)[:, : y.shape[-1]]
    return {"codes": c.to(E4M3), "scales": scale}


def _plain_norm(s):
    case = s["case"]
    R, H, D = case["R"], case.get("H", 1), case["D"]
    h, out = s["x"].float(), {}
    if case["op"] == "quant":
        return _codes(h)
    if case["res"]:
        h = h + s["residual"].float()
        out["residual"] = s["residual"].copy_(h)
    silu = None
    if case["gate"]:
        z = s["gate"].float()
        silu = z / (1 + torch.exp(-z))
    if case["gate"] == "before":
        h = h * silu
    h = h.view(R, H, D)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    y = y.view(R, H * D)
    if case["gate"] == "after":
        y = y * silu
    return {**out, **({"y": y.to(s["x"].dtype)} if case["out"] == "io" else _codes(y))}


def _plain_product(s):
    K, N = s["x"].shape[1], s["w"].shape[0]
    x = s["x"].float() * s["sx"].repeat_interleave(BLOCK, 1)[:, :K]
    sw = s["sw"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    y = torch.matmul(x, (s["w"].float() * sw).t())
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y"].dtype)


def _valid(lens, B, T):
    """[B, T]: whether a row of a padded batch is a token."""
    t = torch.arange(T, device=DEV)
    return (t < lens[:, None]) if lens is not None else t.expand(B, T) >= 0


def _plain_rope(s):
    case = s["case"]
    B, T, Hq, Hkv, D, R = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "R"))
    at = s["pos"][:, None] + torch.arange(T, device=DEV)
    angle = at.double()[..., None] * s["freq"]                  # 64 bits: far positions
    cos, sin = torch.cos(angle).float() * s["magnitude"], torch.sin(angle).float() * s["magnitude"]
    cos, sin = cos[:, :, None], sin[:, :, None]
    ok = _valid(s["lens"], B, T)[:, :, None, None]
    heads = s["x"].view(B, T, Hq + 2 * Hkv, D)
    t = heads[:, :, : Hq + Hkv].float()
    r, rest = t[..., :R], t[..., R:]
    half = case["pairs"] == "half"
    a, b = (r[..., : R // 2], r[..., R // 2:]) if half else (r[..., 0::2], r[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.cat([a, b], -1) if half else torch.stack([a, b], -1).flatten(-2)
    t = torch.cat([r, rest], -1).to(s["x"].dtype)
    parts = {"q": t[:, :, :Hq], "k": t[:, :, Hq:], "v": heads[:, :, Hq + Hkv:]}
    return {n: torch.where(ok, p, 0.0).to(p.dtype) for n, p in parts.items()}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    import gated_delta_rule_40_amd as gdr

    case = s["case"]
    if case["op"] == "norm":
        outs = {n: s[n] for n in ("y", "codes", "scales") if n in s}
        gdr.gdr_rms_norm(s["x"], s["weight"], **outs, residual=s.get("residual"),
                         gate=s.get("gate"), gate_first=case["gate"] == "before", eps=EPS)
        return {**outs, **({"residual": s["residual"]} if case["res"] else {})}
    if case["op"] == "quant":
        gdr.gdr_quant_rows(s["x"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if case["op"] == "product":
        gdr.gdr_matmul_fp8(s["x"], s["sx"], s["w"], s["sw"], s["y"], bias=s["bias"])
        return s["y"]
    gdr.gdr_rope(s["x"], s["freq"], s["pos"], s["q"], s["k"], s["v"], lens=s["lens"],
                 interleaved=case["pairs"] == "interleaved", magnitude=s["magnitude"])
    return {n: s[n] for n in ("q", "k", "v")}


def run(state):
    if own:
        return _own(state)
    plain = {"product": _plain_product, "rope": _plain_rope}
    return plain.get(state["case"]["op"], _plain_norm)(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] in ("norm", "quant"):
        width = case.get("H", 1) * case["D"]
        n = case["R"] * width
        res = {"": 0, "bf16": 4, "f32": 8}[case.get("res", "")]
        out = es if case.get("out") == "io" else 1 + 4 / BLOCK
        return {"bytes": n * (es + res + out + (es if case.get("gate") else 0))
                + (4 * width if case["op"] == "norm" else 0),
                "flops": n * (4 + (5 if case.get("gate") else 0))}
    if case["op"] == "product":
        M, N, K = (case[k] for k in "MNK")
        return {"bytes": M * K + N * K + 4 * (M + N / BLOCK) * (K / BLOCK) + es * M * N,
                "flops": 2.0 * M * N * K}
    # Lengths of padded batches are drawn from the upper half.
    rows = case["B"] * case["T"] * (0.75 if case["ragged"] else 1.0)
    heads = case["Hq"] + 2 * case["Hkv"]
    return {"bytes": 2 * es * rows * heads * case["D"] + 4 * case["R"],
            "flops": rows * (3 * (case["Hq"] + case["Hkv"]) * case["R"] + 10 * case["R"])}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_codes(y):
    """Codes before their rounding (what they stand for), and scales."""
    R, W = y.shape
    nb = -(-W // BLOCK)
    scales = torch.empty(R, nb, dtype=torch.float64, device=DEV)
    codes = torch.empty_like(y)
    for b in range(nb):
        part = y[:, b * BLOCK: (b + 1) * BLOCK]
        scales[:, b] = torch.maximum(part.abs().max(1).values / 448, torch.tensor(2.0 ** -100))
        codes[:, b * BLOCK: (b + 1) * BLOCK] = part / scales[:, b: b + 1]
    return {"codes": codes, "scales": scales}


def _exact_norm(s):
    case = s["case"]
    D = case["D"]
    h, out = s["x"].double(), {}
    if case["op"] == "quant":
        return _exact_codes(h)
    if case["res"]:
        h = h + s["residual"].double()
        out["residual"] = h
    z = s["gate"].double() * torch.sigmoid(s["gate"].double()) if case["gate"] else None
    if case["gate"] == "before":
        h = h * z
    y = torch.empty_like(h)
    for i in range(case["H"]):
        head = h[:, i * D: (i + 1) * D]
        rms = torch.sqrt(torch.linalg.vector_norm(head, dim=1, keepdim=True) ** 2 / D + EPS)
        y[:, i * D: (i + 1) * D] = head / rms * s["weight"][i].double()
    if case["gate"] == "after":
        y = y * z
    return {**out, **({"y": y} if case["out"] == "io" else _exact_codes(y))}


def _exact_product(s):
    """Block by block of the contraction."""
    M, K = s["x"].shape
    N = s["w"].shape[0]
    y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    for b in range(-(-K // BLOCK)):
        at = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        p = s["x"][:, at].double() @ s["w"][:, at].double().t().contiguous()
        col = s["sw"][:, b].double()[torch.arange(N, device=DEV) // BLOCK]
        y += s["sx"][:, b: b + 1].double() * p * col
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_rope(s):
    """Pairs as complex numbers."""
    case = s["case"]
    B, T, Hq, Hkv, D, R = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "R"))
    x = s["x"].double().reshape(B, T, -1, D)
    p = s["pos"].long()[:, None] + torch.arange(T, device=DEV)
    turn = torch.polar(torch.full((B, T, R // 2), s["magnitude"], dtype=torch.float64, device=DEV),
                       p[..., None] * s["freq"])[:, :, None]
    first, second = ((slice(0, R // 2), slice(R // 2, R)) if case["pairs"] == "half"
                     else (slice(0, R, 2), slice(1, R, 2)))
    y = x.clone()
    turned = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y[..., first], y[..., second] = turned.real, turned.imag
    y[:, :, Hq + Hkv:] = x[:, :, Hq + Hkv:]
    for b, n in enumerate([] if s["lens"] is None else s["lens"].tolist()):
        y[b, n:] = 0
    return {"q": y[:, :, :Hq], "k": y[:, :, Hq: Hq + Hkv], "v": y[:, :, Hq + Hkv:]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _exact_product, "rope": _exact_rope}.get(case["op"], _exact_norm)(s)
