"""The 8-bit block-scaled linear: E4M3 codes with one fp32 scale per 128 values of an activation's
row and per 128 x 128 tile of a weight (include/nvfp4.h defines the format).

For the layers a policy keeps out of 4 bits, beside :func:`nvfp4_linear` and with its epilogue:
:func:`fp8_linear` quantizes its bf16 input, :func:`fp8_linear_swiglu` the SwiGLU product of gate
and up, :func:`fp8_gemm` takes codes (from the norms' 8-bit outputs, for one), and
:func:`fp8_linear_train` is differentiable.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import checkpoint as ck
from ._lib import check, lib
from .checkpoint import _rows
from .nvfp4 import (DTYPE_CODES, _activation_code, _epilogue_tensors, _gate_up, _given_workspace, _on_device, _operands,
                    _ptr, _require_cuda, _require_device, _stream, _written)

FP8_BLOCK = 128
FP8_MAX_DIM = 1 << 22


def _blocks(n: int) -> int:
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def _weight(codes: torch.Tensor, scales: torch.Tensor) -> tuple[int, int]:
    """Checks a weight's codes [N, K] and scales [ceil(N/128), ceil(K/128)]; returns N, K."""
    _require_cuda("codes", codes, torch.uint8, 2)
    n, k = codes.shape
    _scales("scales", scales, (_blocks(n), _blocks(k)))
    return n, k


def _scales(name: str, t: torch.Tensor, shape: tuple[int, int]) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous fp32 {list(shape)}, got {getattr(t, 'dtype', None)} "
                         f"{list(getattr(t, 'shape', []))}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")


def _bias(bias: torch.Tensor | None, n: int) -> None:
    if bias is not None:
        _require_cuda("bias", bias, torch.bfloat16)
        if bias.numel() != n:
            raise ValueError(f"bias must have {n} elements, got {bias.numel()}")


def _apart(workspace: torch.Tensor, need: int, *others: torch.Tensor | None) -> None:
    """The ``need`` bytes of a caller's workspace that a call writes (the quantized input, partial
    sums) and reads again share no memory with its operands and outputs."""
    p = workspace.data_ptr()
    for t in others if need else ():
        if t is not None and p < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < p + need:
            raise ValueError("workspace must not overlap the call's operands or outputs")


def fp8_gemm_workspace_bytes(m: int, k: int, n: int) -> int:
    """Workspace fp8_gemm can use to split tiles along K (current device)."""
    return int(lib().nvfp4_fp8_gemm_workspace_bytes(m, k, n))


def fp8_linear_workspace_bytes(m: int, k: int, n: int) -> int:
    """Workspace of fp8_linear for an [m, k] input and n outputs (current device)."""
    return int(lib().nvfp4_fp8_linear_workspace_bytes(m, k, n))


def _empty_codes(rows: int, k: int, device: torch.device) -> tuple[torch.Tensor, torch.Tensor]:
    return (torch.empty(rows, k, dtype=torch.uint8, device=device),
            torch.empty(_blocks(k), rows, dtype=torch.float32, device=device))


@_on_device
def fp8_quantize_activation(x: torch.Tensor, column_sum: bool = False):
    """bf16 [..., K] (K a multiple of 16) to codes uint8 [rows, K] (E4M3) and scales fp32
    [ceil(K/128), rows].  ``column_sum``: also the sums of x over its rows, fp32 [K] (the bias
    gradient of a linear whose output's gradient is x), added in a fixed order."""
    x2, rows, k = _rows("x", x)
    codes, scales = _empty_codes(rows, k, x2.device)
    total, ws, need = None, None, 0
    if column_sum:
        total = torch.empty(k, dtype=torch.float32, device=x2.device)
        need = lib().nvfp4_fp8_quantize_workspace_bytes(rows, k)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x2.device)
    check(lib().nvfp4_fp8_quantize_activation(_ptr(x2), None, rows, k, _ptr(codes), _ptr(scales), _ptr(total), _ptr(ws),
                                              need, _stream(x2.device)))
    return (codes, scales, total) if column_sum else (codes, scales)


@_on_device
def fp8_quantize_checkpoint(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, ck.Checkpoint]:
    """(codes, scales) of fp8_quantize_activation and checkpoint_pack(x), from one read of x."""
    x2, rows, k = _rows("x", x)
    codes, scales = _empty_codes(rows, k, x2.device)
    held = ck._empty_checkpoint(x2)
    check(lib().nvfp4_fp8_quantize_checkpoint(_ptr(x2), rows, k, _ptr(codes), _ptr(scales), _ptr(held.codes),
                                              _ptr(held.scales), _stream(x2.device)))
    return codes, scales, held


@_on_device
def fp8_quantize_swiglu(gate: torch.Tensor, up: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """fp8_quantize_activation(swiglu(gate, up)) without writing the product."""
    g2, u2 = _gate_up(gate, up)
    rows, k = g2.shape
    codes, scales = _empty_codes(rows, k, gate.device)
    check(lib().nvfp4_fp8_quantize_activation(_ptr(g2), _ptr(u2), rows, k, _ptr(codes), _ptr(scales), None, None, 0,
                                              _stream(gate.device)))
    return codes, scales


@_on_device
def fp8_quantize_weight(w: torch.Tensor, transpose: bool = False):
    """bf16 or fp32 weight [N, K] to codes uint8 [N, K] and scales fp32 [ceil(N/128), ceil(K/128)].
    ``transpose``: also the same values as codes [K, N] and scales [ceil(K/128), ceil(N/128)], the
    weight of the input's gradient (N a multiple of 16)."""
    w2, n, k = _rows("weight", w, None)
    if w2.dim() != 2:
        raise ValueError(f"weight must be [out_features, in_features], got shape {list(w.shape)}")
    dev = w2.device
    codes = torch.empty(n, k, dtype=torch.uint8, device=dev)
    scales = torch.empty(_blocks(n), _blocks(k), dtype=torch.float32, device=dev)
    codes_t = scales_t = None
    if transpose:
        codes_t = torch.empty(k, n, dtype=torch.uint8, device=dev)
        scales_t = torch.empty(_blocks(k), _blocks(n), dtype=torch.float32, device=dev)
    check(lib().nvfp4_fp8_quantize_weight(_ptr(w2), DTYPE_CODES[w2.dtype], n, k, _ptr(codes), _ptr(scales), _ptr(codes_t),
                                          _ptr(scales_t), _stream(dev)))
    return (codes, scales, codes_t, scales_t) if transpose else (codes, scales)


@_on_device
def fp8_dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values fp32(code * scale) in ``dtype`` (bf16 or fp32) of an activation's or a weight's
    codes, told apart by the scales' shape."""
    _require_cuda("codes", codes, torch.uint8, 2)
    rows, k = codes.shape
    if dtype not in DTYPE_CODES:
        raise ValueError(f"fp8_dequantize supports bf16 and fp32 outputs, got {dtype}")
    # [ceil(K/128), rows] and [ceil(rows/128), ceil(K/128)] are equal for one row of one block only
    weight = tuple(getattr(scales, "shape", ())) == (_blocks(rows), _blocks(k))
    _scales("scales", scales, (_blocks(rows), _blocks(k)) if weight else (_blocks(k), rows))
    _operands(codes, scales=scales)
    out = torch.empty(rows, k, dtype=dtype, device=codes.device)
    check(lib().nvfp4_fp8_dequantize(_ptr(codes), _ptr(scales), rows, k, int(weight), _ptr(out), DTYPE_CODES[dtype],
                                     _stream(codes.device)))
    return out


@_on_device
def fp8_gemm(x_codes: torch.Tensor, x_scales: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
             bias: torch.Tensor | None = None, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
             activation: str | None = None, residual: torch.Tensor | None = None,
             preact: torch.Tensor | None = None) -> torch.Tensor:
    """The product of an activation's codes [M, K] and a weight's [N, K]: bf16(act(z) + residual)
    from z = product + bias, in fp32 with that one rounding; [M, N].  (The matrix cores add eight
    products at a time, cut below 2^-13 of the largest: 1.4e-5 of the outputs' norm on normal
    values.)  The product of two blocks' scales must be an fp32 number (their largest magnitudes
    multiply to 6.8e43 at most): the output is infinite or NaN otherwise.  ``out``, ``activation``,
    ``residual`` and ``preact`` as for :func:`nvfp4_linear`; the workspace of
    fp8_gemm_workspace_bytes is allocated here if not given.  Outputs may not overlap what the call
    reads, nor a given workspace either."""
    _require_cuda("x_codes", x_codes, torch.uint8, 2)
    m, k = x_codes.shape
    _scales("x_scales", x_scales, (_blocks(k), m))
    n, wk = _weight(codes, scales)
    if wk != k:
        raise ValueError(f"codes must be uint8 [{n}, {k}], got {list(codes.shape)}")
    _bias(bias, n)
    _operands(x_codes, x_scales=x_scales, codes=codes, scales=scales, bias=bias)
    dev = x_codes.device
    act = _activation_code(activation)
    inputs = (x_codes, x_scales, codes, scales) if bias is None else (x_codes, x_scales, codes, scales, bias)
    residual = _epilogue_tensors(m, n, dev, residual, preact, out, *inputs)
    given = out
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    need = fp8_gemm_workspace_bytes(m, k, n)
    if workspace is not None:
        _given_workspace(workspace, dev)
        if workspace.numel() >= need:
            _apart(workspace, need, *inputs, residual, given, preact)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    check(lib().nvfp4_fp8_gemm(_ptr(x_codes), _ptr(x_scales), m, k, _ptr(codes), _ptr(scales), n, _ptr(bias), act,
                               _ptr(residual), _ptr(preact), _ptr(out), _ptr(workspace) if need else None, need,
                               _stream(dev)))
    if given is not None or preact is not None:
        _written(given, preact)
    return out


def _linear(x, x2, up, m, k, codes, scales, bias, workspace, out, activation, residual, preact):
    """fp8_linear of ``x`` (or gate), ``x2`` its checked contiguous rows."""
    n, wk = _weight(codes, scales)
    if wk != k:
        raise ValueError(f"codes must be uint8 [{n}, {k}], got {list(codes.shape)}")
    _bias(bias, n)
    _operands(x, codes=codes, scales=scales, bias=bias)
    dev = x.device
    act = _activation_code(activation)
    given = out
    inputs = (x2, codes, scales, *(t for t in (up, bias) if t is not None))
    if residual is not None or preact is not None or given is not None:
        residual = _epilogue_tensors(m, n, dev, residual, preact, given, *inputs)
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    need = lib().nvfp4_fp8_linear_workspace_bytes(m, k, n)
    if workspace is not None:
        _given_workspace(workspace, dev)
        _apart(workspace, need, *inputs, residual, given, preact)
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    check(lib().nvfp4_fp8_linear(_ptr(x2), _ptr(up), m, k, _ptr(codes), _ptr(scales), _ptr(bias), n, act, _ptr(residual),
                                 _ptr(preact), _ptr(out), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                 _stream(dev)))
    if given is not None or preact is not None:
        _written(given, preact)
    if x.dim() == 2 and (given is None or given.shape == (m, n)):
        return out
    return out.reshape(*x.shape[:-1], n)


@_on_device
def fp8_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, out: torch.Tensor | None = None, activation: str | None = None,
               residual: torch.Tensor | None = None, preact: torch.Tensor | None = None) -> torch.Tensor:
    """The 8-bit block-scaled linear: bf16 x [..., K] quantized to blocks, times the weight's codes
    [N, K]; bf16(act(z) + residual) from z = product + bias, in fp32 with that one rounding.

    ``out``, ``activation``, ``residual`` and ``preact`` as for :func:`nvfp4_linear`."""
    x2, m, k = _rows("x", x)
    return _linear(x, x2, None, m, k, codes, scales, bias, workspace, out, activation, residual, preact)


@_on_device
def fp8_linear_swiglu(gate: torch.Tensor, up: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                      bias: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, activation: str | None = None,
                      residual: torch.Tensor | None = None, preact: torch.Tensor | None = None) -> torch.Tensor:
    """:func:`fp8_linear` on silu(gate) * up, the product never written (down_proj)."""
    g2, u2 = _gate_up(gate, up)
    return _linear(gate, g2, u2, *g2.shape, codes, scales, bias, workspace, out, activation, residual, preact)


class _FP8Fn(torch.autograd.Function):
    """Forward: the master weight's codes, made afresh (it changes every step), and fp8_linear.
    Backward, quantization taken as the identity: the gradient g before the activation is quantized
    to blocks along N and multiplied by the transposed weight codes (grad_x); grad_W = g^T x in bf16,
    g not quantized, x the values of its 8-bit checkpoint (:func:`weight_grad`); grad_b = sum of g
    over rows, taken in the pass that quantizes it.  The residual's gradient is grad_y."""

    @staticmethod
    def forward(ctx, x, weight, bias, x_codes, x_scales, activation, residual):
        n = weight.shape[0]
        w = weight.detach()
        w = w if w.dtype in DTYPE_CODES else w.float()
        codes_t = scales_t = None
        if ctx.needs_input_grad[0]:
            codes, scales, codes_t, scales_t = fp8_quantize_weight(w, transpose=True)
        else:
            codes, scales = fp8_quantize_weight(w)
        b = None if bias is None else bias.detach().to(torch.bfloat16).contiguous()
        z = z_scales = None
        if activation is not None and any(ctx.needs_input_grad[:3]):
            z = torch.empty(x.numel() // x.shape[-1], n, dtype=torch.bfloat16, device=x.device)
        r = None if residual is None else residual.detach()
        if x_codes is None and ctx.needs_input_grad[1]:
            q, s, held = fp8_quantize_checkpoint(x)
            x_codes, x_scales = held.codes, held.scales
            y = fp8_gemm(q, s, codes, scales, b, activation=activation, preact=z, residual=r).reshape(*x.shape[:-1], n)
        else:
            y = fp8_linear(x, codes, scales, b, activation=activation, preact=z, residual=r)
        if z is not None:
            z, z_scales, _ = ck.checkpoint_pack(z)
        if not ctx.needs_input_grad[1]:
            x_codes = x_scales = None
        ctx.save_for_backward(x_codes, x_scales, codes_t, scales_t, z, z_scales)
        ctx.activation = activation
        ctx.shapes = (x.shape, x.dtype, weight.dtype, None if bias is None else bias.dtype,
                      None if residual is None else residual.shape)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x_codes, x_scales, codes_t, scales_t, z, z_scales = ctx.saved_tensors
        x_shape, x_dtype, w_dtype, b_dtype, r_shape = ctx.shapes
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        grad_r = None
        if ctx.needs_input_grad[6]:
            # grad_y itself, which autograd copies into the leaf's gradient while others hold it; a view
            # of it would be kept as the gradient, and added to in place
            grad_r = grad_y if grad_y.shape == r_shape else grad_y.reshape(r_shape).clone()
        g = grad_y.reshape(-1, grad_y.shape[-1])
        if z is not None:
            g = ck.activation_backward(g, ck.Checkpoint(z, z_scales), ctx.activation)
        grad_x = grad_w = grad_b = None
        if need_x or need_b:
            g_codes, g_scales, *total = fp8_quantize_activation(g, column_sum=need_b)
            if need_b:
                grad_b = total[0].to(b_dtype)
            if need_x:
                grad_x = fp8_gemm(g_codes, g_scales, codes_t, scales_t).reshape(x_shape).to(x_dtype)
        if need_w:
            out = w_dtype if w_dtype in DTYPE_CODES else torch.float32
            grad_w = ck.weight_grad(g, ck.Checkpoint(x_codes, x_scales), out).to(w_dtype)
        return grad_x, grad_w, grad_b, None, None, None, grad_r


@_on_device
def fp8_linear_train(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, checkpoint=None,
                     activation: str | None = None, residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable :func:`fp8_linear` on a full-precision master weight [out, in] (``out`` and
    ``in`` multiples of 16), its 8-bit codes made at every call; ``x`` is cast to bf16.

    The output and the input's gradient are products of 8-bit blocks (of the weight with x, and with
    the output's gradient, quantized); the weight's gradient is a bf16 product of the output's
    gradient, not quantized, with the values of x's 8-bit checkpoint (:func:`weight_grad`), which is
    all that is kept of x: ``checkpoint`` shares one (of :func:`layernorm_train`,
    :func:`rmsnorm_train` or :func:`checkpoint_pack`), None packs it here, with x's codes.  Without
    gradients (``torch.no_grad``) it is :func:`fp8_linear`, and keeps nothing.  ``activation`` and
    ``residual`` (bf16, gets its gradient too) as for :func:`nvfp4_linear_train`, the activation's
    gradient at z in 8 bits.

    A backward pass that fills ``.grad`` is captured into a graph only while no eager graph of the
    same leaves is alive: autograd would add on that one's stream, which a capture must not wait for.
    ``torch.autograd.grad`` has no such limit."""
    x = x.to(torch.bfloat16)
    if x.dim() < 1 or not x.is_contiguous():
        x = x.contiguous()
    _activation_code(activation)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.shape[1] != x.shape[-1]:
        raise ValueError(f"weight must be [out_features, {x.shape[-1]}], got {list(getattr(weight, 'shape', []))}")
    if weight.shape[0] % 16:
        raise ValueError(f"fp8_linear_train needs out_features divisible by 16, got {weight.shape[0]}")
    _require_device(x.device, weight=weight, bias=bias, residual=residual)
    codes = scales = None
    if checkpoint is not None:
        if not isinstance(checkpoint, ck.Checkpoint):
            raise TypeError("checkpoint must be None or a Checkpoint")
        codes, scales, rows, k = ck._saved("checkpoint", checkpoint)
        _require_device(x.device, checkpoint=codes)
        if checkpoint.rotation_group or k != x.shape[-1] or rows * k != x.numel():
            raise ValueError(f"checkpoint holds {list(checkpoint.codes.shape)} under rotation group "
                             f"{checkpoint.rotation_group}; the linear's input is {list(x.shape)} without a rotation")
    if not torch.is_grad_enabled():
        # an autograd function is told of leaves that require gradients here too, and would keep for them
        # what no backward pass will read
        layer = FP8Linear.from_weight(weight, bias)
        return layer(x, activation, residual)
    return _FP8Fn.apply(x, weight, bias, codes, scales, activation, residual)


class FP8Linear:
    """An inference linear over a weight in 8-bit blocks, beside :class:`NVFP4Linear`: for the layers
    that keep more than 4 bits.  ``codes`` uint8 (or float8_e4m3fn) [out, in] and ``scales``
    fp32 [ceil(out/128), ceil(in/128)] are E4M3 codes and the factors they are multiplied by."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None):
        if codes.dim() != 2 or codes.shape[1] % 16:
            raise ValueError(f"codes must be [out_features, in_features], in_features a multiple of 16, got "
                             f"{list(codes.shape)}")
        if codes.dtype == torch.float8_e4m3fn:
            codes = codes.view(torch.uint8)
        elif codes.dtype != torch.uint8:
            raise ValueError(f"codes must be uint8 or float8_e4m3fn, got {codes.dtype}")
        self.codes, self.scales, self.bias = codes, scales, bias
        self.out_features, self.in_features = codes.shape
        if tuple(scales.shape) != (_blocks(self.out_features), _blocks(self.in_features)):
            raise ValueError(f"scales must be [{_blocks(self.out_features)}, {_blocks(self.in_features)}], got "
                             f"{list(scales.shape)}")

    @classmethod
    def from_weight(cls, weight: torch.Tensor, bias: torch.Tensor | None = None) -> "FP8Linear":
        """Quantize a full-precision weight [out, in] that lives on the GPU (any float dtype)."""
        w = weight if weight.dtype in DTYPE_CODES else weight.float()
        codes, scales = fp8_quantize_weight(w)
        return cls(codes, scales, None if bias is None else bias.to(torch.bfloat16).contiguous())

    def __call__(self, x: torch.Tensor, activation: str | None = None, residual: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, preact: torch.Tensor | None = None) -> torch.Tensor:
        """The linear on ``x``; the other arguments as in :func:`fp8_linear`."""
        return fp8_linear(x.to(torch.bfloat16), self.codes, self.scales, self.bias, out=out, activation=activation,
                          residual=residual, preact=preact)

    def dequantized_weight(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The weight's values in ``dtype``."""
        return fp8_dequantize(self.codes, self.scales, dtype)
