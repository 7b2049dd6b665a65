"""Layer norm with the residual's addition, in the forms of the RMS norm (norm.py): its output as
bf16, with an 8-bit checkpoint, or as the NVFP4 or 8-bit block codes the linears take; and the RMS
norm's output as 8-bit block codes."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._lib import check, lib
from .checkpoint import Checkpoint, _empty_checkpoint, _rows
from .fp8 import _empty_codes
from .norm import _inputs, _weight
from .nvfp4 import (DTYPE_CODES, _on_device, _ptr, _require_device, _scalar_f32, _stream, scale_bytes,
                    static_global_sf)


def _layer_inputs(x, weight, bias, eps, residual):
    """norm._inputs with the bias behind the weight."""
    args, held, r, rows, k = _inputs(x, weight, eps, residual)
    b = None
    if bias is not None:
        b = _weight(bias, k, x.device)
        if b.dtype != held[2].dtype:
            raise ValueError(f"bias must be of the weight's dtype {held[2].dtype}, got {b.dtype}")
    return (*args[:5], _ptr(b), *args[5:]), (*held, b), r, rows, k


def _layernorm(x, weight, bias, eps, residual, packed: bool):
    args, held, r, _, _ = _layer_inputs(x, weight, bias, eps, residual)
    y = torch.empty_like(held[0], dtype=torch.bfloat16)
    ck = _empty_checkpoint(held[0]) if packed else None
    check(lib().nvfp4_layernorm(*args, _ptr(r), y.data_ptr(), ck.codes.data_ptr() if ck else None,
                                ck.scales.data_ptr() if ck else None, _stream(x.device)))
    return y, r, ck


@_on_device
def layernorm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-6,
              residual: torch.Tensor | None = None):
    """Layer norm over the last dimension (a multiple of 16, at most 16384): bf16 y.

    With ``residual`` the norm is of r = x + residual, and (y, r) is returned, r in the residual's
    dtype.  x, residual and weight are bf16 or fp32 (an fp32 x takes an fp32 residual), bias of the
    weight's dtype; mean and variance are taken in fp64."""
    y, r, _ = _layernorm(x, weight, bias, eps, residual, False)
    return y if residual is None else (y, r)


@_on_device
def layernorm_checkpoint(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-6,
                         residual: torch.Tensor | None = None):
    """:func:`layernorm` with the 8-bit checkpoint of y: (y, checkpoint) or (y, r, checkpoint)."""
    y, r, ck = _layernorm(x, weight, bias, eps, residual, True)
    return (y, ck) if residual is None else (y, r, ck)


@_on_device
def quantize_layernorm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-6,
                       residual: torch.Tensor | None = None, global_sf_x=None):
    """quantize_activation(layernorm(x)) without writing the normed tensor: NVFP4 codes, scales and
    global scale as :func:`nvfp4_gemm` takes them, and with ``residual`` r.  ``global_sf_x=None``:
    dynamic scale."""
    args, _held, r, rows, k = _layer_inputs(x, weight, bias, eps, residual)
    dev = x.device
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(scale_bytes(rows, k), dtype=torch.uint8, device=dev)
    gsf = torch.empty((), dtype=torch.float32, device=dev)
    g, ws, need = None, None, 0
    if global_sf_x is not None:
        g = _scalar_f32(global_sf_x, dev)
        _require_device(dev, global_sf_x=g)
    else:
        need = lib().nvfp4_quantize_layernorm_workspace_bytes(rows)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    if rows == 0:
        # nothing is launched: the scale is the given one, or that of an abs-max of 0
        gsf.copy_(static_global_sf(torch.zeros_like(gsf)) if g is None else g.reshape(()))
    check(lib().nvfp4_quantize_layernorm(*args, _ptr(g), _ptr(r), codes.data_ptr(), scales.data_ptr(), gsf.data_ptr(),
                                         _ptr(ws), need, _stream(dev)))
    return (codes, scales, gsf) if residual is None else (codes, scales, gsf, r)


@_on_device
def fp8_quantize_layernorm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-6,
                           residual: torch.Tensor | None = None):
    """fp8_quantize_activation(layernorm(x)) without writing the normed tensor: 8-bit codes [rows, K]
    and scales as :func:`fp8_gemm` takes them, and with ``residual`` r."""
    args, _held, r, rows, k = _layer_inputs(x, weight, bias, eps, residual)
    codes, scales = _empty_codes(rows, k, x.device)
    check(lib().nvfp4_fp8_quantize_layernorm(*args, _ptr(r), codes.data_ptr(), scales.data_ptr(), _stream(x.device)))
    return (codes, scales) if residual is None else (codes, scales, r)


@_on_device
def fp8_quantize_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                         residual: torch.Tensor | None = None):
    """fp8_quantize_activation(rmsnorm(x)) without writing the normed tensor, as
    :func:`fp8_quantize_layernorm`."""
    args, _held, r, rows, k = _inputs(x, weight, eps, residual)
    codes, scales = _empty_codes(rows, k, x.device)
    check(lib().nvfp4_fp8_quantize_rmsnorm(*args, _ptr(r), codes.data_ptr(), scales.data_ptr(), _stream(x.device)))
    return (codes, scales) if residual is None else (codes, scales, r)


def _layernorm_backward(grad_y, r, weight, eps, grad_residual, parameters: bool):
    """layernorm_backward; without ``parameters`` grad_weight and grad_bias are None."""
    gy, *gm = _rows("grad_y", grad_y)
    r2, rows, k = _rows("r", r, None)
    _require_device(gy.device, r=r, grad_residual=grad_residual)
    if gm != [rows, k]:
        raise ValueError(f"grad_y and r must have the same shape, got {list(grad_y.shape)} and {list(r.shape)}")
    w = _weight(weight, k, gy.device)
    gr = None
    if grad_residual is not None:
        gr, *rm = _rows("grad_residual", grad_residual, r.dtype)
        if rm != [rows, k]:
            raise ValueError(f"grad_residual and r must have the same shape, got {list(grad_residual.shape)} and "
                             f"{list(r.shape)}")
    grad_r = torch.empty_like(r2)
    grad_w = grad_b = ws = None
    if parameters:
        grad_w = torch.empty(k, dtype=torch.float32, device=r2.device)
        grad_b = torch.empty_like(grad_w)
        need = lib().nvfp4_layernorm_backward_workspace_bytes(rows, k)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=r2.device)
    check(lib().nvfp4_layernorm_backward(_ptr(gy), _ptr(r2), DTYPE_CODES[r2.dtype], _ptr(w), DTYPE_CODES[w.dtype],
                                         _ptr(gr), rows, k, float(eps), _ptr(grad_r), _ptr(grad_w), _ptr(grad_b),
                                         _ptr(ws), 0 if ws is None else ws.numel(), _stream(r2.device)))
    return grad_r, grad_w, grad_b


@_on_device
def layernorm_backward(grad_y: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                       grad_residual: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradient of the norm at r (x, or the sum layernorm returned): (grad_r in r's dtype, the
    gradient of x and of the residual alike; grad_weight and grad_bias fp32 [K]).
    ``grad_residual``: the gradient that reaches r along the residual stream, of r's dtype, added
    to grad_r."""
    return _layernorm_backward(grad_y, r, weight, eps, grad_residual, True)


class _LayerNormFn(torch.autograd.Function):
    """y (and r, and y's checkpoint as two non-differentiable byte tensors); keeps r."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps: float, packed: bool):
        y, r, ck = _layernorm_on_device(x, weight, bias, eps, residual, packed)
        ctx.eps = eps
        ctx.has_residual = residual is not None
        ctx.dtypes = (x.dtype, weight.dtype, None if bias is None else bias.dtype)
        ctx.save_for_backward(x if r is None else r, weight)
        ctx.set_materialize_grads(False)
        extra = (ck.codes, ck.scales) if packed else (None, None)
        if packed:
            ctx.mark_non_differentiable(*extra)
        return (y, r, *extra)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_r, _codes, _scales):
        r, weight = ctx.saved_tensors
        xd, wd, bd = ctx.dtypes
        gw = gb = None
        if grad_y is None:
            # only the residual stream was used
            gx = grad_r
        else:
            need_w, need_b = ctx.needs_input_grad[1:3]
            gx, gw, gb = _gradients_on_device(grad_y, r, weight, ctx.eps, grad_r, need_w or need_b)
            gw = gw.to(wd) if need_w else None
            gb = gb.to(bd) if need_b else None
        return (None if gx is None else gx.to(xd), gw, gb, gx if ctx.has_residual else None, None, None)


_layernorm_on_device = _on_device(_layernorm)
_gradients_on_device = _on_device(_layernorm_backward)


def layernorm_train(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-6,
                    residual: torch.Tensor | None = None, checkpoint: bool = False):
    """Differentiable :func:`layernorm`: y, then r with a ``residual``, then with ``checkpoint`` the
    8-bit Checkpoint of y, for the ``checkpoint`` argument of the linears that read y
    (:func:`nvfp4_linear_train`, :func:`fp8_linear_train`)."""
    y, r, codes, scales = _LayerNormFn.apply(x, weight, bias, residual, float(eps), bool(checkpoint))
    out = (y,) if residual is None else (y, r)
    if checkpoint:
        out = (*out, Checkpoint(codes, scales))
    return out if len(out) > 1 else y
