"""Cases for measuring the operators around the NVFP4 linear: the RMS norm with the residual's
addition (quantized to NVFP4, or written with an 8-bit checkpoint, and its gradient), the linear
with activation and residual in its epilogue, and the 8-bit activation checkpoints with the
gradients that read them.

Number formats, as include/nvfp4.h defines them.  NVFP4: E2M1 codes two per byte (even index in
the low nibble), one E4M3 scale per 16 values stored as [ceil(K/128)][rows][8], one fp32 global
scale 2688 / amax.  Checkpoint: E4M3 codes, one power-of-two scale byte (2^(byte - 127)) per 32
values of a row, the smallest power that brings the block's abs-max to 448 or below.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
MIN_EXP, MAX_EXP = -110, 120      # exponents of a checkpoint's block scales


def listed():
    return [
        # one new token between two blocks of a 5120-wide model: the residual's addition, the
        # norm and the dynamic NVFP4 quantization that feeds the projections
        {"name": "norm_nvfp4_decode", "op": "norm_nvfp4", "m": 1, "k": 5120, "stream": "bf16", "static": False},
        # the same at prefill, where it moves activation-sized arrays
        {"name": "norm_nvfp4_prefill", "op": "norm_nvfp4", "m": 4096, "k": 5120, "stream": "bf16", "static": False},
        # training forward over an odd number of rows: fp32 residual stream, bf16 output for the
        # forward projections and its 8-bit checkpoint for their weight gradients
        {"name": "norm_checkpoint", "op": "norm_checkpoint", "m": 4091, "k": 5120, "stream": "f32"},
        # the norm's gradient, with the gradient that arrives along the residual stream
        {"name": "norm_backward", "op": "norm_backward", "m": 4096, "k": 5120, "stream": "bf16"},
        # attention output projection of one token, added to the residual stream
        {"name": "linear_o_proj_decode", "op": "linear", "m": 1, "k": 8192, "n": 5120, "act": "none", "bias": False,
         "residual": True, "group": 0},
        # down projection of 16 sequences' tokens from gate and up, added to the residual stream
        {"name": "linear_down_decode", "op": "linear_swiglu", "m": 16, "k": 25600, "n": 5120, "residual": True},
        # a vision block's first feed-forward linear (rotated input) over an odd number of rows
        {"name": "linear_fc_in", "op": "linear", "m": 4091, "k": 1024, "n": 4096, "act": "gelu", "bias": True,
         "residual": False, "group": 16},
        # the largest feed-forward product at prefill, with bias and activation
        {"name": "linear_ffn_prefill", "op": "linear", "m": 4096, "k": 5120, "n": 25600, "act": "gelu_tanh",
         "bias": True, "residual": False, "group": 0},
        # SwiGLU in a training forward: the product, and gate and up kept in 8 bits
        {"name": "swiglu_checkpoint", "op": "swiglu_checkpoint", "m": 4096, "k": 25600},
        # SwiGLU's gradient from the 8-bit gate and up
        {"name": "swiglu_backward", "op": "swiglu_backward", "m": 4096, "k": 25600},
        # weight gradient of the gate projection from its 8-bit input
        {"name": "weight_grad_gate", "op": "weight_grad", "m": 4096, "n": 25600, "k": 5120, "group": 0, "pack": False},
        # a narrow projection over a short ragged batch: rotate, pack and use the checkpoint
        {"name": "weight_grad_k_proj", "op": "weight_grad", "m": 777, "n": 1024, "k": 5120, "group": 16, "pack": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_nvfp4", "norm_checkpoint", "norm_backward", "linear", "linear", "linear_swiglu",
                     "swiglu_checkpoint", "swiglu_backward", "weight_grad", "weight_grad"])
    m = _log_int(rng, 1, 4096)
    k = 16 * _log_int(rng, 8, 512)
    if op in ("norm_nvfp4", "norm_checkpoint", "norm_backward"):
        case = {"op": op, "m": m, "k": k, "stream": rng.choice(["bf16", "f32"])}
        if op == "norm_nvfp4":
            case["static"] = rng.random() < 0.5
        return case
    if op in ("swiglu_checkpoint", "swiglu_backward"):
        return {"op": op, "m": m, "k": 16 * _log_int(rng, 8, 1600)}
    n = _log_int(rng, 16, 8192)
    if op == "linear_swiglu":
        return {"op": op, "m": m, "k": k, "n": n, "residual": rng.random() < 0.5}
    group = 16 if rng.random() < 0.3 else 0
    if op == "linear":
        return {"op": op, "m": m, "k": k, "n": n, "act": rng.choice(["none", "gelu", "gelu_tanh", "silu"]),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "group": group}
    return {"op": op, "m": m, "n": n, "k": k, "group": group, "pack": group > 0 or rng.random() < 0.5}


# ---- number formats in elementary torch operations (fp32) ----

def _const(v, like):
    # a device scalar: dividing by or into it is an IEEE division, which a Python scalar's is not
    return torch.full((), float(v), dtype=torch.float32, device=like.device)


def _e2m1(a):
    """|a| to the nearest E2M1 magnitude, ties to the even code, 6 at most."""
    half = torch.round(2.0 * a) * 0.5
    return torch.where(a < 2.0, half, torch.where(a < 4.0, torch.round(a), torch.round(a * 0.5) * 2.0)).clamp(max=6.0)


def _nvfp4(v, gsf):
    """fp32 [rows, K] -> E2M1 values and E4M3 scales, both as fp32: [rows, K], [rows, K/16]."""
    b = v.reshape(v.shape[0], -1, 16)
    s = (gsf * b.abs().amax(-1) / _const(6.0, v)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    r = torch.where(s > 0, gsf / s, torch.zeros_like(s))
    q = b * r[..., None]
    return (_e2m1(q.abs()) * torch.sign(q)).reshape(v.shape), s


def _global_scale(v):
    return _const(2688.0, v) / v.abs().amax().clamp(min=1e-12)


def _rotate(v, g):
    """Block Hadamard rotation of fp32 rows, butterflies of growing stride, rounded to bf16."""
    if not g:
        return v
    b = v.reshape(-1, g)
    h = 1
    while h < g:
        p = b.reshape(-1, g // (2 * h), 2, h)
        b = torch.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), 2).reshape(-1, g)
        h *= 2
    return (b * float(torch.tensor(1.0 / math.sqrt(g), dtype=torch.float32))).to(torch.bfloat16).float().reshape(v.shape)


def _pack_layout(s):
    """Block scales [rows, K/16] (fp32 values) -> library layout bytes."""
    rows, nb = s.shape
    kt = (nb + 7) // 8
    p = torch.zeros((rows, kt * 8), dtype=torch.uint8, device=s.device)
    p[:, :nb] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return p.reshape(rows, kt, 8).permute(1, 0, 2).contiguous().reshape(-1)


def _unpack_layout(b, rows, k, dtype=torch.float32):
    kt = (k + 127) // 128
    s = b.reshape(kt, rows, 8).permute(1, 0, 2).reshape(rows, kt * 8)[:, :k // 16].contiguous()
    return s.view(torch.float8_e4m3fn).to(dtype)


def _pack_codes(q):
    """E2M1 values -> packed bytes."""
    a = q.abs()
    mag = torch.where(a < 2.0, 2.0 * a, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)).to(torch.uint8)
    c = mag | (torch.signbit(q).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _unpack_codes(p, dtype=torch.float32):
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=p.device)
    return torch.stack((lut[(p & 15).long()], lut[(p >> 4).long()]), -1).reshape(p.shape[0], -1)


def _weight(n, k, gen):
    w = (0.02 * torch.randn((n, k), generator=gen, device=DEV)).to(torch.bfloat16).float()
    gsf = _global_scale(w)
    q, s = _nvfp4(w, gsf)
    return _pack_codes(q), _pack_layout(s), gsf


def _blocks32(v):
    pad = -v.shape[1] % 32
    return torch.nn.functional.pad(v, (0, pad)).reshape(v.shape[0], -1, 32)


def _checkpoint(v):
    """fp32 [rows, K] -> E4M3 codes [rows, K] and scale bytes [rows, ceil(K/32)]."""
    b = _blocks32(v)
    mant, e = torch.frexp(b.abs().amax(-1))          # abs-max = mant 2^e, 448 = 0.875 2^9
    e = e - 9 + (mant > 0.875).to(e.dtype)
    e = torch.where(mant == 0, torch.full_like(e, MIN_EXP), e).clamp(MIN_EXP, MAX_EXP)
    c = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn)
    return c.reshape(v.shape[0], -1)[:, :v.shape[1]].contiguous(), (e + 127).to(torch.uint8)


def _checkpoint_values(codes, scales, dtype=torch.float32):
    k = codes.shape[1]
    s = torch.exp2(scales.to(dtype) - 127.0).repeat_interleave(32, 1)[:, :k]
    return codes.to(dtype) * s


# ---- inputs ----

def _randn(shape, gen, dtype=torch.bfloat16, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device=DEV)).to(dtype)


def _activations(shape, gen, dtype=torch.bfloat16):
    """Normal values, one in a hundred twenty times larger: activations with outliers."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.01, 20.0 * x, x).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, m, k = case["op"], case["m"], case["k"]
    s = {"case": case}
    if op.startswith("norm"):
        stream = torch.bfloat16 if case["stream"] == "bf16" else torch.float32
        s["w"] = 1.0 + _randn((k,), gen, torch.float32, 0.1)
        if op == "norm_backward":
            s["r"] = _activations((m, k), gen, stream)
            s["gy"] = _randn((m, k), gen, scale=1e-2)
            s["gr"] = _randn((m, k), gen, stream, 1e-2)
            return s
        s["x"], s["res"] = _randn((m, k), gen), _activations((m, k), gen, stream)
        if op == "norm_nvfp4":
            s["gsf"] = _const(2688.0 / 24.0, s["x"]) if case["static"] else None
        return s
    if op in ("linear", "linear_swiglu"):
        n = case["n"]
        if op == "linear":
            s["x"] = _activations((m, k), gen)
            s["bias"] = _randn((n,), gen, scale=0.1) if case["bias"] else None
        else:
            s["gate"], s["up"] = _randn((m, k), gen), _randn((m, k), gen)
        s["packed"], s["scale"], s["gsf_w"] = _weight(n, k, gen)
        s["res"] = _randn((m, n), gen) if case["residual"] else None
        return s
    if op == "swiglu_checkpoint":
        s["gate"], s["up"] = _randn((m, k), gen), _randn((m, k), gen)
        return s
    if op == "swiglu_backward":
        s["gate"], s["up"] = _checkpoint(_randn((m, k), gen).float()), _checkpoint(_randn((m, k), gen).float())
        s["gy"] = _randn((m, k), gen, scale=1e-2)
        return s
    s["gy"] = _randn((m, case["n"]), gen, scale=1e-2)
    x = _activations((m, k), gen)
    s["x"] = x if case["pack"] else _checkpoint(x.float())
    return s


# ---- one pass ----

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import nvfp4_w4a4_quantized_global_amd as nv
    c = s["case"]
    op = c["op"]
    if op == "norm_nvfp4":
        codes, scales, gsf, r = nv.quantize_rmsnorm(s["x"], s["w"], EPS, s["res"], s["gsf"])
        return nv.dequantize(codes, scales, gsf), gsf, r
    if op == "norm_checkpoint":
        y, r, ck = nv.rmsnorm_checkpoint(s["x"], s["w"], EPS, s["res"])
        return y, r, ck.codes.view(torch.float8_e4m3fn), ck.scales
    if op == "norm_backward":
        return nv.rmsnorm_backward(s["gy"], s["r"], s["w"], EPS, s["gr"])
    if op == "linear":
        act = None if c["act"] == "none" else c["act"]
        return nv.nvfp4_linear(s["x"], s["packed"], s["scale"], s["gsf_w"], s["bias"], c["n"], None, c["group"],
                               activation=act, residual=s["res"])
    if op == "linear_swiglu":
        return nv.nvfp4_linear_swiglu(s["gate"], s["up"], s["packed"], s["scale"], s["gsf_w"], None, c["n"],
                                      residual=s["res"])
    if op == "swiglu_checkpoint":
        x, g, u = nv.swiglu_checkpoint(s["gate"], s["up"])
        return x, g.codes.view(torch.float8_e4m3fn), g.scales, u.codes.view(torch.float8_e4m3fn), u.scales
    if op == "swiglu_backward":
        gate, up = (nv.Checkpoint(a.view(torch.uint8), b) for a, b in (s["gate"], s["up"]))
        return nv.swiglu_backward(s["gy"], gate, up)
    ck = nv.checkpoint_pack(s["x"], c["group"]) if c["pack"] else nv.Checkpoint(s["x"][0].view(torch.uint8), s["x"][1])
    return nv.weight_grad(s["gy"], ck)


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _norm(x, res, w):
    r = (x.float() + res.float()).to(res.dtype)
    # the mean square in 64 bits: its rounding to 32 decides codes next to a border
    scale = (r.double().square().mean(-1, keepdim=True) + EPS).rsqrt().float()
    return r, (r.float() * scale * w.float()).to(torch.bfloat16)


def _product(x, packed, scale, gsf_w, n, k):
    """alpha * (x quantized) (packed)^T in fp32, x fp32 [rows, K] already rotated."""
    gsf = _global_scale(x)
    q, sx = _nvfp4(x, gsf)
    a = q * sx.repeat_interleave(16, 1)
    b = _unpack_codes(packed) * _unpack_layout(scale, n, k).repeat_interleave(16, 1)
    return torch.matmul(a, b.t()) * (_const(1.0, x) / (gsf * gsf_w))


def _plain(s):
    c = s["case"]
    op, k = c["op"], c["k"]
    if op == "norm_nvfp4":
        r, y = _norm(s["x"], s["res"], s["w"])
        y = y.float()
        gsf = _global_scale(y) if s["gsf"] is None else s["gsf"]
        q, sc = _nvfp4(y, gsf)
        return (q * sc.repeat_interleave(16, 1) / gsf).to(torch.bfloat16), gsf, r
    if op == "norm_checkpoint":
        r, y = _norm(s["x"], s["res"], s["w"])
        return (y, r) + _checkpoint(y.float())
    if op == "norm_backward":
        r, gy = s["r"].float(), s["gy"].float()
        rs = (r.double().square().mean(-1, keepdim=True) + EPS).rsqrt().float()
        gw = gy * s["w"]
        dot = (gw * r).sum(-1, keepdim=True) / k
        gx = gw * rs - r * (rs * rs * rs * dot) + s["gr"].float()
        return gx.to(s["r"].dtype), (gy * (r * rs)).sum(0)
    if op == "linear":
        z = _product(_rotate(s["x"].float(), c["group"]), s["packed"], s["scale"], s["gsf_w"], c["n"], k)
        if s["bias"] is not None:
            z = z + s["bias"].float()
        z = _act(z, c["act"])
        return (z if s["res"] is None else z + s["res"].float()).to(torch.bfloat16)
    if op in ("linear_swiglu", "swiglu_checkpoint"):
        g, u = s["gate"].float(), s["up"].float()
        x = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
        if op == "swiglu_checkpoint":
            return (x,) + _checkpoint(g) + _checkpoint(u)
        z = _product(x.float(), s["packed"], s["scale"], s["gsf_w"], c["n"], k)
        return (z if s["res"] is None else z + s["res"].float()).to(torch.bfloat16)
    gy = s["gy"].float()
    if op == "swiglu_backward":
        g, u = _checkpoint_values(*s["gate"]), _checkpoint_values(*s["up"])
        sg = 1.0 / (1.0 + torch.exp(-g))
        return (gy * u * sg * (1.0 + g * (1.0 - sg))).to(torch.bfloat16), (gy * g * sg).to(torch.bfloat16)
    codes, scales = _checkpoint(_rotate(s["x"].float(), c["group"])) if c["pack"] else s["x"]
    return torch.matmul(gy.t(), _checkpoint_values(codes, scales))


# ---- the definitions in 64 bits ----

def _f32(v):
    """One rounding to fp32, back in 64 bits (where the format prescribes it)."""
    return v.float().double()


def _to_grid(v, grid):
    """Magnitudes to the nearest entry of an ascending grid, ties to the even index, saturating."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, v), torch.searchsorted(mid, v, right=True)
    return torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))


def _grid_e2m1():
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)


def _grid_e4m3():
    sub = [i * 2.0 ** -9 for i in range(8)]
    return torch.tensor(sub + [(1 + i / 8) * 2.0 ** (e - 7) for e in range(1, 16) for i in range(8)][:-1],
                        dtype=torch.float64, device=DEV)


def _exact_gsf(v):
    return _f32(2688.0 / v.abs().max().clamp(min=float(torch.tensor(1e-12, dtype=torch.float32))))


def _exact_nvfp4(v, gsf):
    """code * scale of every value of v (64 bits, values of bf16)."""
    b = v.reshape(v.shape[0], v.shape[1] // 16, 16)
    e4 = _grid_e4m3()
    s = e4[_to_grid(_f32(_f32(gsf * b.abs().max(-1).values) / 6.0), e4)].unsqueeze(-1)
    p = _f32(b * _f32(gsf / s.clamp(min=2.0 ** -9)))
    mag = _grid_e2m1()[_to_grid(p.abs(), _grid_e2m1())]
    return (torch.where(p < 0, -mag, mag) * s).reshape(v.shape)


def _exact_hadamard(v, g):
    if not g:
        return v
    i = torch.arange(g, device=DEV)
    bits = i[:, None] & i[None, :]
    parity = sum((bits >> j) & 1 for j in range(g.bit_length())) % 2
    h = (1.0 - 2.0 * parity.double()) / math.sqrt(g)
    return (v.reshape(-1, g) @ h).reshape(v.shape).to(torch.bfloat16).double()


def _exact_checkpoint(v):
    """codes (values, 64 bits) and block exponents + 127."""
    rows, k = v.shape
    nb = (k + 31) // 32
    b = torch.zeros((rows, nb * 32), dtype=torch.float64, device=DEV)
    b[:, :k] = v
    b = b.reshape(rows, nb, 32)
    top = b.abs().max(-1).values
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(MIN_EXP, MAX_EXP)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where((top <= 224.0 * torch.exp2(e)) & (e > MIN_EXP), e - 1, e))
    p = b / torch.exp2(e).unsqueeze(-1)
    g = _grid_e4m3()
    mag = g[_to_grid(p.abs().contiguous(), g)]
    return torch.where(p < 0, -mag, mag).reshape(rows, -1)[:, :k], (e + 127).to(torch.uint8), e


def _exact_values(ck):
    codes, scales = ck
    e = scales.double() - 127.0
    k = codes.shape[1]
    return codes.double() * torch.exp2(e)[:, torch.arange(k, device=DEV) // 32]


def _exact_linear(x, s, c, act, bias, res):
    gsf = _exact_gsf(x)
    a = _exact_nvfp4(x, gsf)
    n, k = c["n"], c["k"]
    b = _unpack_codes(s["packed"], torch.float64)
    b = b * _unpack_layout(s["scale"], n, k, torch.float64)[:, torch.arange(k, device=DEV) // 16]
    z = a.matmul(b.t()) / (gsf * s["gsf_w"].double())
    if bias is not None:
        z = z + bias.double()
    if act == "gelu":
        z = z * torch.special.erfc(-z / math.sqrt(2.0)) / 2.0
    elif act == "gelu_tanh":
        z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    elif act == "silu":
        z = z * torch.sigmoid(z)
    return z if res is None else z + res.double()


def exact(case, seed):
    s = prepare(case, seed)
    op, k = case["op"], case["k"]
    if op in ("norm_nvfp4", "norm_checkpoint"):
        t = s["x"].double() + s["res"].double()
        r = t.to(s["res"].dtype).double()
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / k + EPS) * s["w"].double()
        yb = y.to(torch.bfloat16).double()
        if op == "norm_nvfp4":
            gsf = _exact_gsf(yb) if s["gsf"] is None else s["gsf"].double()
            return _exact_nvfp4(yb, gsf) / gsf, gsf, t
        codes, scales, _ = _exact_checkpoint(yb)
        return y, t, codes, scales
    if op == "norm_backward":
        r, gy, w = s["r"].double(), s["gy"].double(), s["w"].double()
        rs = 1.0 / torch.sqrt((r * r).sum(1, keepdim=True) / k + EPS)
        n = r * rs
        gn = gy * w
        return rs * (gn - n * (gn * n).mean(1, keepdim=True)) + s["gr"].double(), (gy * n).sum(0)
    if op == "linear":
        return _exact_linear(_exact_hadamard(s["x"].double(), case["group"]), s, case, case["act"], s["bias"], s["res"])
    if op in ("linear_swiglu", "swiglu_checkpoint"):
        g, u = s["gate"].double(), s["up"].double()
        x = g * torch.sigmoid(g) * u
        if op == "linear_swiglu":
            return _exact_linear(x.to(torch.bfloat16).double(), s, case, "none", None, s["res"])
        cg, cu = _exact_checkpoint(g), _exact_checkpoint(u)
        return x, cg[0], cg[1], cu[0], cu[1]
    gy = s["gy"].double()
    if op == "swiglu_backward":
        g, u = _exact_values(s["gate"]), _exact_values(s["up"])
        sg = torch.sigmoid(g)
        return gy * u * (sg + g * sg * (1.0 - sg)), gy * g * sg
    if case["pack"]:
        codes, scales, _ = _exact_checkpoint(_exact_hadamard(s["x"].double(), case["group"]))
        return gy.t().contiguous().matmul(_exact_values((codes, scales)))
    return gy.t().contiguous().matmul(_exact_values(s["x"]))


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    mk = m * k
    if op.startswith("norm"):
        st = 2 if case["stream"] == "bf16" else 4
        if op == "norm_backward":         # gradient, stream and its gradient in; gradient out
            return {"bytes": mk * (2 + 3 * st) + 8 * k, "flops": 12 * mk}
        out = mk / 2 + mk / 16 + 2 * mk if op == "norm_nvfp4" else 2 * mk + mk + mk / 32
        return {"bytes": mk * (2 + 2 * st) + out + 4 * k, "flops": 8 * mk}
    if op in ("linear", "linear_swiglu"):
        n = case["n"]
        w = n * k * (0.5 + 1 / 16)
        x = 2 * mk if op == "linear" else 4 * mk
        return {"bytes": w + x + 2 * m * n * (2 if case["residual"] else 1), "flops": 2.0 * mk * n}
    if op == "swiglu_checkpoint":
        return {"bytes": mk * (4 + 2) + 2 * mk * (1 + 1 / 32), "flops": 10 * mk}
    if op == "swiglu_backward":
        return {"bytes": mk * (2 + 4) + 2 * mk * (1 + 1 / 32), "flops": 12 * mk}
    n = case["n"]
    x = 2 * mk if case["pack"] else mk * (1 + 1 / 32)
    return {"bytes": x + 2 * m * n + 4 * n * k, "flops": 2.0 * mk * n}
