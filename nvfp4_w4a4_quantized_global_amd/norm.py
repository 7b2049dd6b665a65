"""RMS norm with the residual's addition: the step before a block's linears, with its
output as bf16, with an 8-bit checkpoint, or as the NVFP4 codes the linears take."""
from __future__ import annotations

import torch

from ._lib import check, lib
from .checkpoint import Checkpoint, _empty_checkpoint, _rows
from .nvfp4 import (DTYPE_CODES, _on_device, _ptr, _require_device, _scalar_f32, _stream, scale_bytes,
                    static_global_sf)

NORM_MAX_K = 16384


def _stream_rows(name: str, t: torch.Tensor) -> tuple[torch.Tensor, int, int]:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in DTYPE_CODES:
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return _rows(name, t, t.dtype)


def _weight(weight: torch.Tensor, k: int, device: torch.device) -> torch.Tensor:
    w, rows, n = _stream_rows("weight", weight)
    if n != k or rows != 1 or w.dim() != 1:
        raise ValueError(f"weight must be bf16 or fp32 [{k}], got {weight.dtype} {list(weight.shape)}")
    _require_device(device, weight=w)
    return w


class _Inputs:
    """The checked inputs of one norm call, in the order of the C calls' first arguments."""

    def __init__(self, x, weight, eps, residual):
        self.x, self.rows, self.k = _stream_rows("x", x)
        self.w = _weight(weight, self.k, x.device)
        self.res = self.out = None
        if residual is not None:
            self.res, _, _ = _stream_rows("residual", residual)
            _require_device(x.device, residual=residual)
            if residual.shape != x.shape:
                raise ValueError(f"x and residual must have the same shape, got {list(x.shape)} and "
                                 f"{list(residual.shape)}")
            if x.dtype == torch.float32 and residual.dtype != torch.float32:
                raise ValueError("an fp32 x needs an fp32 residual")
            self.out = x.new_empty(x.shape, dtype=self.res.dtype)
        self.args = (_ptr(self.x), DTYPE_CODES[x.dtype], _ptr(self.res),
                     DTYPE_CODES[x.dtype if self.res is None else self.res.dtype], _ptr(self.w),
                     DTYPE_CODES[self.w.dtype], self.rows, self.k, float(eps))


def _rmsnorm(x, weight, eps, residual, packed: bool):
    a = _Inputs(x, weight, eps, residual)
    y = x.new_empty(x.shape, dtype=torch.bfloat16)
    ck = _empty_checkpoint(x) if packed else None
    check(lib().nvfp4_rmsnorm(*a.args, _ptr(a.out), _ptr(y), _ptr(ck.codes) if ck else None,
                              _ptr(ck.scales) if ck else None, _stream(x.device)))
    return y, a.out, ck


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
    a = _Inputs(x, weight, eps, residual)
    dev = x.device
    codes = x.new_empty((a.rows, a.k // 2), dtype=torch.uint8)
    scales = x.new_empty((scale_bytes(a.rows, a.k),), dtype=torch.uint8)
    gsf = x.new_empty((), dtype=torch.float32)
    g = None if global_sf_x is None else _scalar_f32(global_sf_x, dev)
    _require_device(dev, global_sf_x=g)
    if a.rows == 0:
        # nothing is launched: the scale is the given one, or that of an abs-max of 0
        gsf.copy_(static_global_sf(torch.zeros_like(gsf)) if g is None else g.reshape(()))
    need = lib().nvfp4_quantize_rmsnorm_workspace_bytes(a.rows) if g is None else 0
    ws = x.new_empty((need,), dtype=torch.uint8) if need else None
    check(lib().nvfp4_quantize_rmsnorm(*a.args, _ptr(g), _ptr(a.out), _ptr(codes), _ptr(scales), _ptr(gsf), _ptr(ws),
                                       need, _stream(dev)))
    return (codes, scales, gsf) if residual is None else (codes, scales, gsf, a.out)


@_on_device
def rmsnorm_backward(grad_y: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                     grad_residual: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of the norm at r (x, or the sum rmsnorm returned): (grad_r in r's dtype, the
    gradient of x and of the residual alike; grad_weight fp32 [K]).  ``grad_residual``: the
    gradient that reaches r along the residual stream, of r's dtype, added to grad_r."""
    gy, *gm = _rows("grad_y", grad_y)
    r2, rows, k = _stream_rows("r", r)
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
    grad_r = r.new_empty(r.shape)
    grad_w = r.new_empty((k,), dtype=torch.float32)
    need = lib().nvfp4_rmsnorm_backward_workspace_bytes(rows, k)
    ws = r.new_empty((max(need, 256),), dtype=torch.uint8)
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
