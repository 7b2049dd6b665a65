"""8-bit activation checkpoints and the gradients that read them.

A training forward keeps its activations for the backward; :func:`checkpoint_pack` keeps a
bf16 tensor as E4M3 codes with one power-of-two scale byte per 32 values (include/nvfp4.h
defines the format), and :func:`weight_grad`, :func:`swiglu_backward` and
:func:`activation_backward` compute from that form directly.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from ._lib import check, lib
from .nvfp4 import (DTYPE_CODES, _activation_code, _gate_up, _on_device, _ptr, _require_device, _stream)

CHECKPOINT_BLOCK = 32


class Checkpoint(NamedTuple):
    """An activation in 8 bits: ``codes`` uint8 [..., K] (E4M3), ``scales`` uint8
    [..., ceil(K/32)] (the power of two 2^(byte - 127) of each 32 values), and the rotation
    group under which it was packed (0 = none)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rotation_group: int = 0

    def dequantized(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The values, in bf16 (exact) or fp32."""
        return checkpoint_unpack(self, dtype)


def _scale_columns(k: int) -> int:
    return (k + CHECKPOINT_BLOCK - 1) // CHECKPOINT_BLOCK


def _rows(name: str, t: torch.Tensor, dtype: torch.dtype | None = torch.bfloat16) -> tuple[torch.Tensor, int, int]:
    """``t`` [..., K] of ``dtype`` (None: bf16 or fp32) as contiguous 16-byte aligned rows on a
    GPU (copied where its strides or address differ), with the number of rows and K."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype and (dtype is not None or t.dtype not in DTYPE_CODES):
        raise ValueError(f"{name} must be {dtype or 'bf16 or fp32'}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    k = t.shape[-1]
    rows = t.numel() // k if k else 0
    if not t.is_contiguous():
        t = t.contiguous()
    if t.data_ptr() % 16:
        t = t.clone(memory_format=torch.contiguous_format)
    return t, rows, k


def _saved(name: str, ck: Checkpoint) -> tuple[torch.Tensor, torch.Tensor, int, int]:
    """A checkpoint's codes and scales as contiguous rows, checked, with the rows and K."""
    codes, rows, k = _rows(f"{name}.codes", ck.codes, torch.uint8)
    scales, cols = ck.scales, _scale_columns(k)
    if scales.dtype != torch.uint8 or scales.device != codes.device or scales.numel() != rows * cols \
            or scales.shape[-1:] != (cols,):
        raise ValueError(f"{name}.scales must be uint8 with {rows} rows of {cols} on {codes.device}, got "
                         f"{scales.dtype} {list(scales.shape)} on {scales.device}")
    return codes, scales if scales.is_contiguous() else scales.contiguous(), rows, k


# New tensors come from empty_like on a contiguous tensor of their shape, or from sizes given
# one by one: each some 0.5 us less host time than new_empty with a shape.
def _empty_checkpoint(x: torch.Tensor, rotation_group: int = 0) -> Checkpoint:
    """Room for the checkpoint of x (contiguous)."""
    *lead, k = x.shape
    return Checkpoint(torch.empty_like(x, dtype=torch.uint8),
                      torch.empty(*lead, _scale_columns(k), dtype=torch.uint8, device=x.device), rotation_group)


@_on_device
def checkpoint_pack(x: torch.Tensor, rotation_group: int = 0) -> Checkpoint:
    """bf16 [..., K] (K a multiple of 16) to its 8-bit checkpoint, after the optional block
    rotation.  A value moves by at most 2^-4 of itself, or 2^-10 of its 32 values' power of two
    where that is more; infinities and NaN become NaN."""
    x2, rows, k = _rows("x", x)
    ck = _empty_checkpoint(x2, int(rotation_group))
    check(lib().nvfp4_checkpoint_pack(_ptr(x2), rows, k, int(rotation_group), _ptr(ck.codes), _ptr(ck.scales),
                                      _stream(x.device)))
    return ck


def checkpoint_unpack(ck: Checkpoint, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """A checkpoint's values (still rotated if it was packed so), in bf16 (exact) or fp32."""
    return _unpack(ck.codes, ck, dtype)


@_on_device
def _unpack(_device_of: torch.Tensor, ck: Checkpoint, dtype: torch.dtype) -> torch.Tensor:
    if dtype not in DTYPE_CODES:
        raise ValueError(f"checkpoint_unpack supports bf16 and fp32 outputs, got {dtype}")
    codes, scales, rows, k = _saved("checkpoint", ck)
    out = torch.empty(ck.codes.shape, dtype=dtype, device=codes.device)
    check(lib().nvfp4_checkpoint_unpack(_ptr(codes), _ptr(scales), rows, k, _ptr(out), DTYPE_CODES[dtype],
                                        _stream(codes.device)))
    return out


@_on_device
def weight_grad(grad_y: torch.Tensor, ck: Checkpoint, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The weight gradient of a linear from the checkpoint of its input: grad_y^T x, [N, K],
    for grad_y bf16 [..., N] and x [..., K].  Products are exact, sums fp32; ``dtype`` is the
    result's (fp32 or bf16).  The same inputs give the same bits."""
    gy, m, n = _rows("grad_y", grad_y)
    if dtype not in DTYPE_CODES:
        raise ValueError(f"weight_grad supports fp32 and bf16 results, got {dtype}")
    codes, scales, rows, k = _saved("checkpoint", ck)
    _require_device(gy.device, checkpoint=codes)
    if rows != m:
        raise ValueError(f"grad_y has {m} rows, the checkpoint {rows}")
    out = torch.empty(n, k, dtype=dtype, device=gy.device)
    need = lib().nvfp4_weight_grad_workspace_bytes(m, n, k)
    ws = torch.empty(need, dtype=torch.uint8, device=gy.device) if need else None
    check(lib().nvfp4_weight_grad(_ptr(gy), m, n, _ptr(codes), _ptr(scales), k, _ptr(out), DTYPE_CODES[dtype], _ptr(ws),
                                  need, _stream(gy.device)))
    return out


@_on_device
def swiglu_checkpoint(gate: torch.Tensor, up: torch.Tensor) -> tuple[torch.Tensor, Checkpoint, Checkpoint]:
    """:func:`swiglu` and the 8-bit checkpoints of ``gate`` and ``up``, in one pass."""
    g2, u2 = _gate_up(gate, up)
    like = g2 if gate.dim() == 2 else g2.view(gate.shape)
    x = torch.empty_like(like)
    g, u = _empty_checkpoint(like), _empty_checkpoint(like)
    check(lib().nvfp4_swiglu_checkpoint(_ptr(g2), _ptr(u2), g2.shape[0], g2.shape[1], _ptr(x), _ptr(g.codes),
                                        _ptr(g.scales), _ptr(u.codes), _ptr(u.scales), _stream(gate.device)))
    return x, g, u


@_on_device
def swiglu_backward(grad_x: torch.Tensor, gate, up) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradients (bf16) of :func:`swiglu` at ``gate`` and ``up``: both Checkpoints, or both
    bf16 tensors, of grad_x's shape."""
    gx, rows, k = _rows("grad_x", grad_x)
    packed = isinstance(gate, Checkpoint)
    if packed != isinstance(up, Checkpoint):
        raise ValueError("gate and up must be both checkpoints or both bf16 tensors")
    if packed:
        if gate.rotation_group or up.rotation_group:
            raise ValueError("gate and up must be packed without a rotation")
        (g, gs, *gm), (u, us, *um) = _saved("gate", gate), _saved("up", up)
    else:
        gs = us = None
        (g, *gm), (u, *um) = _rows("gate", gate), _rows("up", up)
    _require_device(gx.device, gate=g, up=u)
    if gm != [rows, k] or um != [rows, k]:
        raise ValueError(f"grad_x, gate and up must have the same shape, got {list(gx.shape)}, {list(g.shape)} and "
                         f"{list(u.shape)}")
    dg, du = torch.empty_like(gx), torch.empty_like(gx)
    check(lib().nvfp4_swiglu_backward(_ptr(gx), _ptr(g), _ptr(gs), _ptr(u), _ptr(us), rows, k, _ptr(dg), _ptr(du),
                                      _stream(gx.device)))
    return dg, du


@_on_device
def activation_backward(grad_y: torch.Tensor, z, activation: str | None) -> torch.Tensor:
    """bf16(grad_y act'(z)): the gradient before the activation of a linear's epilogue.  ``z``:
    its ``preact`` (bf16, any width), or that tensor's Checkpoint."""
    gy, rows, n = _rows("grad_y", grad_y)
    act = _activation_code(activation)
    if isinstance(z, Checkpoint):
        if z.rotation_group:
            raise ValueError("z must be packed without a rotation")
        z2, zs, *zm = _saved("z", z)
    else:
        zs = None
        z2, *zm = _rows("z", z)
    _require_device(gy.device, z=z2)
    if zm != [rows, n]:
        raise ValueError(f"grad_y and z must have the same shape, got {list(gy.shape)} and {list(z2.shape)}")
    out = torch.empty_like(gy)
    check(lib().nvfp4_activation_backward(_ptr(gy), _ptr(z2), _ptr(zs), rows, n, act, _ptr(out), _stream(gy.device)))
    return out


class _SwiGLUFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, checkpoint: bool):
        from .nvfp4 import swiglu
        ctx.packed = checkpoint
        if checkpoint:
            x, g, u = swiglu_checkpoint(gate, up)
            ctx.save_for_backward(g.codes, g.scales, u.codes, u.scales)
        else:
            x = swiglu(gate, up)
            ctx.save_for_backward(gate, up)
        return x

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_x):
        if ctx.packed:
            gc, gs, uc, us = ctx.saved_tensors
            gate, up = Checkpoint(gc, gs), Checkpoint(uc, us)
        else:
            gate, up = ctx.saved_tensors
        return (*swiglu_backward(grad_x, gate, up), None)


def swiglu_train(gate: torch.Tensor, up: torch.Tensor, checkpoint: bool = False) -> torch.Tensor:
    """Differentiable :func:`swiglu` (bf16).  ``checkpoint``: keep gate and up for the
    backward in 8 bits, and take the gradients at those values."""
    return _SwiGLUFn.apply(gate, up, bool(checkpoint))


