"""Cases for measuring the layer norm (its output as bf16 with an 8-bit checkpoint, as 8-bit
block codes or as NVFP4 codes, and its gradient) and the 8-bit block-scaled linear (one token,
a few, many, with its epilogue, and a training step).

Number formats, as include/nvfp4.h defines them.  8-bit blocks: E4M3 codes, one fp32 scale per
128 values of an activation row (stored [ceil(K/128)][rows]) and per 128 x 128 tile of a weight
([ceil(N/128)][ceil(K/128)]), scale = largest magnitude / 448.  Checkpoint: E4M3 codes, one
power-of-two scale byte (2^(byte - 127)) per 32 values of a row, the smallest power that brings
the block's abs-max to 448 or below.  NVFP4: E2M1 codes two per byte, one E4M3 scale per 16
values, one fp32 global scale 2688 / amax.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = 128
FLOOR = 448.0 * 2.0 ** -110       # smallest abs-max a block's scale is made from
MIN_EXP, MAX_EXP = -110, 120      # exponents of a checkpoint's block scales


def listed():
    return [
        # one new token before a block's 8-bit projections: the residual's addition and the norm
        {"name": "layernorm_fp8_decode", "op": "layernorm_fp8", "m": 1, "k": 5120, "stream": "bf16", "bias": True},
        # a vision block's norm over an odd number of rows, fp32 residual stream, 8-bit projections
        {"name": "layernorm_fp8_vision", "op": "layernorm_fp8", "m": 4091, "k": 1024, "stream": "f32", "bias": True},
        # a prefill in front of 4-bit projections with a dynamic scale
        {"name": "layernorm_nvfp4_prefill", "op": "layernorm_nvfp4", "m": 4096, "k": 5120, "stream": "bf16",
         "bias": True},
        # training forward of a vision block over eight tiles of 2048 rows: bf16 output for the
        # projections and its 8-bit checkpoint for their weight gradients
        {"name": "layernorm_checkpoint", "op": "layernorm_checkpoint", "m": 16384, "k": 1024, "stream": "bf16",
         "bias": True},
        # the norm's gradient over the same tiles, with the gradient along the residual stream
        {"name": "layernorm_backward_vision", "op": "layernorm_backward", "m": 16384, "k": 1024, "stream": "bf16"},
        # the same of a wide model with an fp32 stream and an odd number of rows
        {"name": "layernorm_backward_wide", "op": "layernorm_backward", "m": 4091, "k": 5120, "stream": "f32"},
        # attention output projection of one token, added to the residual stream
        {"name": "fp8_o_proj_decode", "op": "fp8_linear", "m": 1, "k": 8192, "n": 5120, "act": "none", "bias": False,
         "residual": True},
        # down projection of 16 sequences' tokens, kept in 8 bits, from gate and up
        {"name": "fp8_down_decode", "op": "fp8_linear_swiglu", "m": 16, "k": 25600, "n": 5120, "residual": True},
        # a small ragged batch through odd widths: K that is no whole number of blocks, odd N
        {"name": "fp8_ragged", "op": "fp8_linear", "m": 777, "k": 1040, "n": 1001, "act": "silu", "bias": True,
         "residual": False},
        # a vision block's first feed-forward linear over an odd number of rows
        {"name": "fp8_fc_in", "op": "fp8_linear", "m": 4091, "k": 1024, "n": 4096, "act": "gelu", "bias": True,
         "residual": False},
        # the largest feed-forward product at prefill
        {"name": "fp8_gate_prefill", "op": "fp8_linear", "m": 4096, "k": 5120, "n": 25600, "act": "none",
         "bias": False, "residual": False},
        # a training step of a query projection: output, and the gradients of input, weight and bias
        {"name": "fp8_train", "op": "fp8_train", "m": 4096, "k": 5120, "n": 8192},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layernorm_fp8", "layernorm_nvfp4", "layernorm_checkpoint", "layernorm_backward", "fp8_linear",
                     "fp8_linear", "fp8_linear", "fp8_linear_swiglu", "fp8_train"])
    m = _log_int(rng, 1, 4096)
    k = 16 * _log_int(rng, 8, 512)
    if op.startswith("layernorm"):
        case = {"op": op, "m": m, "k": k, "stream": rng.choice(["bf16", "f32"])}
        if op != "layernorm_backward":
            case["bias"] = rng.random() < 0.7
        return case
    if op == "fp8_train":
        return {"op": op, "m": m, "k": k, "n": 16 * _log_int(rng, 8, 512)}
    n = _log_int(rng, 16, 8192)
    if op == "fp8_linear_swiglu":
        return {"op": op, "m": m, "k": k, "n": n, "residual": rng.random() < 0.5}
    return {"op": op, "m": m, "k": k, "n": n, "act": rng.choice(["none", "gelu", "gelu_tanh", "silu"]),
            "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}


# ---- number formats in elementary torch operations (fp32) ----

def _const(v, like):
    # a device scalar: dividing by or into it is an IEEE division, which a Python scalar's is not
    return torch.full((), float(v), dtype=torch.float32, device=like.device)


def _pad(v, rows, cols):
    return torch.nn.functional.pad(v, (0, -v.shape[1] % cols, 0, -v.shape[0] % rows))


def _fp8_blocks(v, rows):
    """fp32 [M, K] -> E4M3 codes [M, K] and fp32 scales [ceil(M/rows), ceil(K/128)] of tiles of
    rows x 128."""
    p = _pad(v, rows, BLOCK)
    b = p.reshape(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)
    top = torch.maximum(b.abs().amax((1, 3)), _const(FLOOR, v))
    r = _const(448.0, v) / top
    q = (b * r[:, None, :, None]).to(torch.float8_e4m3fn).reshape(p.shape)
    return q[:v.shape[0], :v.shape[1]].contiguous(), top / _const(448.0, v)


def _fp8_values(codes, scales, rows, dtype=torch.float32):
    s = scales.to(dtype).repeat_interleave(rows, 0)[:codes.shape[0]].repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.to(dtype) * s


def _e2m1(a):
    """|a| to the nearest E2M1 magnitude, ties to the even code, 6 at most."""
    half = torch.round(2.0 * a) * 0.5
    return torch.where(a < 2.0, half, torch.where(a < 4.0, torch.round(a), torch.round(a * 0.5) * 2.0)).clamp(max=6.0)


def _nvfp4(v, gsf):
    """fp32 [rows, K] -> the values its codes and scales stand for, times the global scale."""
    b = v.reshape(v.shape[0], -1, 16)
    s = (gsf * b.abs().amax(-1) / _const(6.0, v)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    q = b * torch.where(s > 0, gsf / s, torch.zeros_like(s))[..., None]
    return (_e2m1(q.abs()) * torch.sign(q) * s[..., None]).reshape(v.shape)


def _checkpoint(v):
    """fp32 [rows, K] -> E4M3 codes [rows, K] and scale bytes [rows, ceil(K/32)]."""
    b = _pad(v, 1, 32)
    b = b.reshape(b.shape[0], -1, 32)
    mant, e = torch.frexp(b.abs().amax(-1))          # abs-max = mant 2^e, 448 = 0.875 2^9
    e = e - 9 + (mant > 0.875).to(e.dtype)
    e = torch.where(mant == 0, torch.full_like(e, MIN_EXP), e).clamp(MIN_EXP, MAX_EXP)
    c = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn)
    return c.reshape(v.shape[0], -1)[:, :v.shape[1]].contiguous(), (e + 127).to(torch.uint8)


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
    if op.startswith("layernorm"):
        stream = torch.bfloat16 if case["stream"] == "bf16" else torch.float32
        s["w"] = 1.0 + _randn((k,), gen, torch.float32, 0.1)
        # rows whose mean is not zero
        s["res"] = _activations((m, k), gen, stream) + _randn((m, 1), gen, stream)
        if op == "layernorm_backward":
            s["gy"] = _randn((m, k), gen, scale=1e-2)
            s["gr"] = _randn((m, k), gen, stream, 1e-2)
            return s
        s["x"] = _randn((m, k), gen)
        s["b"] = _randn((k,), gen, torch.float32, 0.1) if case["bias"] else None
        return s
    n = case["n"]
    if op == "fp8_train":
        s["x"] = _activations((m, k), gen).requires_grad_()
        s["w"] = _randn((n, k), gen, torch.float32, 0.02).requires_grad_()
        s["bias"] = _randn((n,), gen, torch.float32, 0.1).requires_grad_()
        s["gy"] = _randn((m, n), gen, scale=1e-2)
        return s
    if op == "fp8_linear":
        s["x"] = _activations((m, k), gen)
        s["bias"] = _randn((n,), gen, scale=0.1) if case["bias"] else None
    else:
        s["gate"], s["up"] = _randn((m, k), gen), _randn((m, k), gen)
        s["bias"] = None
    s["codes"], s["scales"] = _fp8_blocks(_randn((n, k), gen, scale=0.02).float(), BLOCK)
    s["res"] = _randn((m, n), gen) if case["residual"] else None
    return s


# ---- one pass ----

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import nvfp4_w4a4_quantized_global_amd as nv
    c = s["case"]
    op = c["op"]
    if op == "layernorm_fp8":
        codes, scales, r = nv.fp8_quantize_layernorm(s["x"], s["w"], s["b"], EPS, s["res"])
        return codes.view(torch.float8_e4m3fn), scales, r
    if op == "layernorm_nvfp4":
        codes, scales, gsf, r = nv.quantize_layernorm(s["x"], s["w"], s["b"], EPS, s["res"])
        return nv.dequantize(codes, scales, gsf), gsf, r
    if op == "layernorm_checkpoint":
        y, r, ck = nv.layernorm_checkpoint(s["x"], s["w"], s["b"], EPS, s["res"])
        return y, r, ck.codes.view(torch.float8_e4m3fn), ck.scales
    if op == "layernorm_backward":
        return nv.layernorm_backward(s["gy"], s["res"], s["w"], EPS, s["gr"])
    if op == "fp8_train":
        y = nv.fp8_linear_train(s["x"], s["w"], s["bias"])
        return (y.detach(), *torch.autograd.grad(y, (s["x"], s["w"], s["bias"]), s["gy"]))
    w = s["codes"].view(torch.uint8)
    if op == "fp8_linear":
        act = None if c["act"] == "none" else c["act"]
        return nv.fp8_linear(s["x"], w, s["scales"], s["bias"], activation=act, residual=s["res"])
    return nv.fp8_linear_swiglu(s["gate"], s["up"], w, s["scales"], residual=s["res"])


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _statistics(r):
    # mean and variance in 64 bits: their rounding to 32 decides codes next to a border
    d = r.double()
    c = d - d.mean(-1, keepdim=True)
    return c, (c.square().mean(-1, keepdim=True) + EPS).rsqrt()


def _layernorm(x, res, w, b):
    r = (x.float() + res.float()).to(res.dtype)
    c, s = _statistics(r)
    y = c.float() * s.float() * w
    return r, (y if b is None else y + b).to(torch.bfloat16)


def _product(x, codes, scales):
    q, s = _fp8_blocks(x, 1)
    return torch.matmul(_fp8_values(q, s, 1), _fp8_values(codes, scales, BLOCK).t())


def _plain(s):
    c = s["case"]
    op, k = c["op"], c["k"]
    if op == "layernorm_backward":
        d, rs = _statistics(s["res"])
        n, gy = (d * rs).float(), s["gy"].float()
        g = gy * s["w"]
        gx = rs.float() * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) + s["gr"].float()
        return gx.to(s["res"].dtype), (gy * n).sum(0), gy.sum(0)
    if op.startswith("layernorm"):
        r, y = _layernorm(s["x"], s["res"], s["w"], s["b"])
        if op == "layernorm_fp8":
            codes, scales = _fp8_blocks(y.float(), 1)
            return codes, scales.t().contiguous(), r
        y32 = y.float()
        if op == "layernorm_nvfp4":
            gsf = _const(2688.0, y) / y32.abs().amax().clamp(min=1e-12)
            return (_nvfp4(y32, gsf) / gsf).to(torch.bfloat16), gsf, r
        return (y, r) + _checkpoint(y32)
    if op == "fp8_train":
        x, w, gy = s["x"].detach().float(), s["w"].detach(), s["gy"].float()
        codes, scales = _fp8_blocks(w, BLOCK)
        y = (_product(x, codes, scales) + s["bias"].detach().to(torch.bfloat16).float()).to(torch.bfloat16)
        q, sg = _fp8_blocks(gy, 1)
        gx = torch.matmul(_fp8_values(q, sg, 1), _fp8_values(codes, scales, BLOCK)).to(torch.bfloat16)
        kept, e = _checkpoint(x)
        xv = kept.float() * torch.exp2(e.float() - 127.0).repeat_interleave(32, 1)[:, :k]
        return y, gx, torch.matmul(gy.t(), xv), gy.sum(0)
    if op == "fp8_linear":
        x = s["x"].float()
    else:
        g, u = s["gate"].float(), s["up"].float()
        x = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16).float()
    z = _product(x, s["codes"], s["scales"])
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = _act(z, c.get("act"))
    return (z if s["res"] is None else z + s["res"].float()).to(torch.bfloat16)


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


def _round_e4m3(p):
    g = _grid_e4m3()
    mag = g[_to_grid(p.abs().contiguous(), g)]
    return torch.where(p < 0, -mag, mag)


def _exact_fp8(v, rows):
    """codes (values) and scales, 64 bits, of tiles of rows x 128 cut one column of tiles at a time."""
    codes, scales = torch.empty_like(v), []
    for c0 in range(0, v.shape[1], BLOCK):
        col = v[:, c0:c0 + BLOCK]
        tops = [t.abs().max() for t in col.split(rows)] if rows > 1 else [col.abs().max(1).values]
        top = torch.stack([t.reshape(-1) for t in tops]).reshape(-1).clamp(min=FLOOR)
        each = top.repeat_interleave(rows)[:v.shape[0], None]
        codes[:, c0:c0 + BLOCK] = _round_e4m3(_f32(col * _f32(448.0 / each)))
        scales.append(_f32(top / 448.0))
    return codes, torch.stack(scales, 1)


def _exact_expand(codes, scales, rows):
    i, j = (torch.arange(n, device=DEV) for n in codes.shape)
    return codes.double() * scales.double()[(i // rows)[:, None], (j // BLOCK)[None, :]]


def _exact_checkpoint(v):
    """codes (values, 64 bits) and block exponents."""
    rows, k = v.shape
    b = torch.zeros((rows, (k + 31) // 32 * 32), dtype=torch.float64, device=DEV)
    b[:, :k] = v
    b = b.reshape(rows, -1, 32)
    top = b.abs().max(-1).values
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(MIN_EXP, MAX_EXP)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where((top <= 224.0 * torch.exp2(e)) & (e > MIN_EXP), e - 1, e))
    return _round_e4m3(b / torch.exp2(e)[..., None]).reshape(rows, -1)[:, :k], e


def _exact_norm(r):
    mu = r.sum(1, keepdim=True) / r.shape[1]
    rs = 1.0 / torch.sqrt(((r - mu) ** 2).sum(1, keepdim=True) / r.shape[1] + EPS)
    return (r - mu) * rs, rs


def exact(case, seed):
    s = prepare(case, seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "layernorm_backward":
        n, rs = _exact_norm(s["res"].double())
        gy = s["gy"].double()
        g = gy * s["w"].double()
        gx = rs * (g - g.sum(1, keepdim=True) / k - n * ((g * n).sum(1, keepdim=True) / k)) + s["gr"].double()
        return gx, (gy * n).sum(0), gy.sum(0)
    if op.startswith("layernorm"):
        t = s["x"].double() + s["res"].double()
        y = _exact_norm(t.to(s["res"].dtype).double())[0] * s["w"].double()
        if s["b"] is not None:
            y = y + s["b"].double()
        yb = y.to(torch.bfloat16).double()
        if op == "layernorm_fp8":
            codes, scales = _exact_fp8(yb, 1)
            return codes, scales.t().contiguous(), t
        if op == "layernorm_checkpoint":
            codes, e = _exact_checkpoint(yb)
            return y, t, codes, (e + 127).to(torch.uint8)
        gsf = _f32(2688.0 / yb.abs().max().clamp(min=float(torch.tensor(1e-12, dtype=torch.float32))))
        b = yb.reshape(m, k // 16, 16)
        sc = _round_e4m3(_f32(_f32(gsf * b.abs().max(-1).values) / 6.0)).unsqueeze(-1)
        p = _f32(b * _f32(gsf / sc.clamp(min=2.0 ** -9)))
        mag = _grid_e2m1()[_to_grid(p.abs(), _grid_e2m1())]
        return (torch.where(p < 0, -mag, mag) * sc).reshape(m, k) / gsf, gsf, t
    if op == "fp8_train":
        x, gy = s["x"].detach().double(), s["gy"].double()
        w = _exact_expand(*_exact_fp8(s["w"].detach().double(), BLOCK), BLOCK)
        y = _exact_expand(*_exact_fp8(x, 1), 1).matmul(w.t()) + s["bias"].detach().to(torch.bfloat16).double()
        gx = _exact_expand(*_exact_fp8(gy, 1), 1).matmul(w)
        codes, e = _exact_checkpoint(x)
        xv = codes * torch.exp2(e)[:, torch.arange(k, device=DEV) // 32]
        return y, gx, gy.t().contiguous().matmul(xv), gy.sum(0)
    if op == "fp8_linear":
        x = s["x"].double()
    else:
        g = s["gate"].double()
        x = (g * torch.sigmoid(g) * s["up"].double()).to(torch.bfloat16).double()
    z = _exact_expand(*_exact_fp8(x, 1), 1).matmul(_exact_expand(s["codes"], s["scales"], BLOCK).t())
    if s["bias"] is not None:
        z = z + s["bias"].double()
    act = case.get("act")
    if act == "gelu":
        z = z * torch.special.erfc(-z / math.sqrt(2.0)) / 2.0
    elif act == "gelu_tanh":
        z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    elif act == "silu":
        z = z * torch.sigmoid(z)
    return z if s["res"] is None else z + s["res"].double()


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    mk = m * k
    if op.startswith("layernorm"):
        st = 2 if case["stream"] == "bf16" else 4
        if op == "layernorm_backward":        # gradient, stream and its gradient in; gradient out
            return {"bytes": mk * (2 + 3 * st) + 12 * k, "flops": 16 * mk}
        out = {"layernorm_fp8": 1 + 4 / BLOCK, "layernorm_nvfp4": 0.5 + 1 / 16 + 2,
               "layernorm_checkpoint": 2 + 1 + 1 / 32}[op]
        return {"bytes": mk * (2 + 2 * st + out) + 8 * k, "flops": 10 * mk}
    n = case["n"]
    if op == "fp8_train":       # x, weight and the output's gradient in; output and the gradients out
        return {"bytes": 4 * mk + 8 * n * k + 4 * m * n + 8 * n, "flops": 6.0 * mk * n}
    x = 4 * mk if op == "fp8_linear_swiglu" else 2 * mk
    return {"bytes": n * k + x + 2 * m * n * (2 if case["residual"] else 1), "flops": 2.0 * mk * n}
