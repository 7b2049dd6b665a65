"""RMS norm with the residual's addition: the step before a block's linears, with its
output as bf16, with an 8-bit checkpoint, or as the NVFP4 codes the linears take."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._lib import check, lib
from .checkpoint import Checkpoint, _empty_checkpoint, _rows
from .nvfp4 import (DTYPE_CODES, _on_device, _ptr, _require_device, _scalar_f32, _stream, scale_bytes,
                    static_global_sf)

NORM_MAX_K = 16384


def _weight(weight: torch.Tensor, k: int, device: torch.device) -> torch.Tensor:
    w, rows, n = _rows("weight", weight, None)
    if n != k or rows != 1 or w.dim() != 1:
        raise ValueError(f"weight must be bf16 or fp32 [{k}], got {weight.dtype} {list(weight.shape)}")
    if w.device != device:
        raise ValueError(f"weight must be on {device}, got {w.device}")
    return w


def _inputs(x, weight, eps, residual):
    """The checked inputs of one norm call in the order of the C calls' first arguments, the
    tensors behind them (which may be copies), r's tensor (None without a residual), rows, K."""
    x2, rows, k = _rows("x", x, None)
    w = _weight(weight, k, x.device)
    xd = rd = DTYPE_CODES[x.dtype]
    r2 = out = None
    if residual is not None:
        r2, _, _ = _rows("residual", residual, None)
        if r2.device != x.device:
            raise ValueError(f"residual must be on {x.device}, got {r2.device}")
        if residual.shape != x.shape:
            raise ValueError(f"x and residual must have the same shape, got {list(x.shape)} and {list(residual.shape)}")
        if x.dtype == torch.float32 and residual.dtype != torch.float32:
            raise ValueError("an fp32 x needs an fp32 residual")
        rd = DTYPE_CODES[residual.dtype]
        out = torch.empty_like(x2, dtype=residual.dtype)
    args = (x2.data_ptr(), xd, _ptr(r2), rd, w.data_ptr(), DTYPE_CODES[w.dtype], rows, k, float(eps))
    return args, (x2, r2, w), out, rows, k


def _rmsnorm(x, weight, eps, residual, packed: bool):
    args, held, r, _, _ = _inputs(x, weight, eps, residual)
    y = torch.empty_like(held[0], dtype=torch.bfloat16)
    ck = _empty_checkpoint(held[0]) if packed else None
    check(lib().nvfp4_rmsnorm(*args, _ptr(r), y.data_ptr(), ck.codes.data_ptr() if ck else None,
                              ck.scales.data_ptr() if ck else None, _stream(x.device)))
    return y, r, ck


@_on_device
def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None):
    """RMS norm over the last dimension (a multiple of 16, at most 16384): bf16 y.

    With ``residual`` the norm is of r = x + residual, and (y, r) is returned, r in the
    residual's dtype.  x, residual and weight are bf16 or fp32 (an fp32 x takes an fp32
    residual); the mean square is summed in fp64."""
    y, r, _ = _rmsnorm(x, weight, eps, residual, False)
    return y if residual is None else (y, r)


@_on_device
def rmsnorm_checkpoint(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None):
    """:func:`rmsnorm` with the 8-bit checkpoint of y: (y, checkpoint) or (y, r, checkpoint)."""
    y, r, ck = _rmsnorm(x, weight, eps, residual, True)
    return (y, ck) if residual is None else (y, r, ck)


@_on_device
def quantize_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                     global_sf_x=None):
    """quantize_activation(rmsnorm(x)) without writing the normed tensor: codes uint8
    [rows, K/2], scales (library layout) and the global scale, as :func:`nvfp4_gemm` takes
    them; with ``residual`` also r.  ``global_sf_x=None``: dynamic scale."""
    args, _held, r, rows, k = _inputs(x, weight, eps, residual)
    dev = x.device
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(scale_bytes(rows, k), dtype=torch.uint8, device=dev)
    gsf = torch.empty((), dtype=torch.float32, device=dev)
    g, ws, need = None, None, 0
    if global_sf_x is not None:
        g = _scalar_f32(global_sf_x, dev)
        _require_device(dev, global_sf_x=g)
    else:
        need = lib().nvfp4_quantize_rmsnorm_workspace_bytes(rows)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    if rows == 0:
        # nothing is launched: the scale is the given one, or that of an abs-max of 0
        gsf.copy_(static_global_sf(torch.zeros_like(gsf)) if g is None else g.reshape(()))
    check(lib().nvfp4_quantize_rmsnorm(*args, _ptr(g), _ptr(r), codes.data_ptr(), scales.data_ptr(), gsf.data_ptr(),
                                       _ptr(ws), need, _stream(dev)))
    return (codes, scales, gsf) if residual is None else (codes, scales, gsf, r)


@_on_device
def rmsnorm_backward(grad_y: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                     grad_residual: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of the norm at r (x, or the sum rmsnorm returned): (grad_r in r's dtype, the
    gradient of x and of the residual alike; grad_weight fp32 [K]).  ``grad_residual``: the
    gradient that reaches r along the residual stream, of r's dtype, added to grad_r."""
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
    grad_w = torch.empty(k, dtype=torch.float32, device=r.device)
    need = lib().nvfp4_rmsnorm_backward_workspace_bytes(rows, k)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=r.device)
    check(lib().nvfp4_rmsnorm_backward(_ptr(gy), _ptr(r2), DTYPE_CODES[r.dtype], _ptr(w), DTYPE_CODES[w.dtype], _ptr(gr),
                                       rows, k, float(eps), _ptr(grad_r), _ptr(grad_w), _ptr(ws), ws.numel(),
                                       _stream(r.device)))
    return grad_r, grad_w


class _RMSNormFn(torch.autograd.Function):
    """y (and r, and y's checkpoint as two non-differentiable byte tensors); keeps r."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps: float, packed: bool):
        y, r, ck = _rmsnorm_on_device(x, weight, eps, residual, packed)
        ctx.eps = eps
        ctx.has_residual = residual is not None
        ctx.dtypes = (x.dtype, weight.dtype)
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
        if grad_y is None:
            # only the residual stream was used
            gx, gw = grad_r, None
        else:
            gx, gw = rmsnorm_backward(grad_y, r, weight, ctx.eps, grad_r)
            gw = gw.to(ctx.dtypes[1])
        return (None if gx is None else gx.to(ctx.dtypes[0]), gw, gx if ctx.has_residual else None, None, None)


_rmsnorm_on_device = _on_device(_rmsnorm)


def rmsnorm_train(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                  checkpoint: bool = False):
    """Differentiable :func:`rmsnorm`: y, then r with a ``residual``, then with
    ``checkpoint`` the 8-bit Checkpoint of y, for the ``checkpoint`` argument of the
    linears that read y (:func:`nvfp4_linear_train`)."""
    y, r, codes, scales = _RMSNormFn.apply(x, weight, residual, float(eps), bool(checkpoint))
    out = (y,) if residual is None else (y, r)
    if checkpoint:
        out = (*out, Checkpoint(codes, scales))
    return out if len(out) > 1 else y
