"""Plain definitions of the operators around the linear: the RMS norm and its gradient, the
8-bit checkpoint format, the epilogue's activations and the gradients that read checkpoints.

Real-valued steps are float64; where the contract fixes a rounding (the norm's scale and
output, the checkpoint's codes) it is applied explicitly.  Pins: tests/test_oracle_operators.py.
"""
from __future__ import annotations

import math

import numpy as np

from .nvfp4 import bf16_round, e4m3_decode

__all__ = ["rmsnorm", "rmsnorm_grads", "checkpoint_pack", "checkpoint_unpack", "activation", "activation_grad",
           "silu_grads"]

CK_BLOCK = 32
CK_MIN_EXP, CK_MAX_EXP = -110, 120


def _f32(a):
    return np.asarray(a, dtype=np.float64).astype(np.float32)


def rmsnorm(x, weight, eps, residual=None, stream: str = "bf16") -> tuple[np.ndarray, np.ndarray]:
    """(r, y): r = x + residual in fp32, rounded to the stream's type; y =
    bf16(fp32(fp32(r * s) * w)) with s = fp32(1 / sqrt(mean(r^2) + eps)).  eps is the fp32
    value the C call receives."""
    r = _f32(x)
    if residual is not None:
        r = (r + _f32(residual)).astype(np.float32)
        if stream == "bf16":
            r = bf16_round(r)
    ms = np.sum(r.astype(np.float64) ** 2, axis=-1, keepdims=True) / r.shape[-1]
    s = _f32(1.0 / np.sqrt(ms + np.float64(np.float32(eps))))
    return r, bf16_round(((r * s).astype(np.float32) * _f32(weight)).astype(np.float32))


def rmsnorm_grads(grad_y, r, weight, eps, grad_residual=None) -> tuple[np.ndarray, np.ndarray]:
    """float64 gradients of y = r w / sqrt(mean(r^2) + eps) for r and w."""
    r, gy, w = (np.asarray(a, dtype=np.float64) for a in (r, grad_y, weight))
    s = 1.0 / np.sqrt(np.mean(r * r, axis=-1, keepdims=True) + np.float64(np.float32(eps)))
    g = gy * w
    grad_r = s * g - r * s ** 3 * np.mean(g * r, axis=-1, keepdims=True)
    if grad_residual is not None:
        grad_r = grad_r + np.asarray(grad_residual, dtype=np.float64)
    return grad_r, np.sum(gy * r * s, axis=0)


def checkpoint_pack(x) -> tuple[np.ndarray, np.ndarray]:
    """uint8 codes [rows, K] and scale bytes [rows, ceil(K/32)], by search: the smallest
    exponent whose 448 multiple holds the block, then the nearest E4M3 value (ties to the
    even code)."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    nb = -(-k // CK_BLOCK)
    p = np.zeros((rows, nb * CK_BLOCK))
    p[:, :k] = x
    p = p.reshape(rows, nb, CK_BLOCK)
    fine = np.isfinite(p)
    top = np.max(np.where(fine, np.abs(p), 0.0), axis=-1)
    exps = np.arange(CK_MIN_EXP, CK_MAX_EXP + 1)
    e = exps[np.minimum(np.searchsorted(448.0 * 2.0 ** exps.astype(np.float64), top), len(exps) - 1)]
    grid = e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.where(fine, p, 0.0) / 2.0 ** e[..., None].astype(np.float64)
    lo = np.searchsorted(mid, np.abs(v), side="left")
    hi = np.searchsorted(mid, np.abs(v), side="right")
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo).astype(np.uint8)
    code = np.where(fine, code | (np.signbit(p).astype(np.uint8) << 7), np.uint8(0x7F))
    return np.ascontiguousarray(code.reshape(rows, -1)[:, :k]), (e + 127).astype(np.uint8)


def checkpoint_unpack(codes, scales) -> np.ndarray:
    """float64 values (NaN codes as NaN)."""
    codes = np.asarray(codes, dtype=np.uint8)
    mag = codes & 0x7F
    v = np.where(mag == 0x7F, np.nan, e4m3_decode(np.minimum(mag, 126)).astype(np.float64))
    v = np.where(codes & 0x80, -v, v)
    s = 2.0 ** (np.asarray(scales).astype(np.float64) - 127.0)
    return v * np.repeat(s, CK_BLOCK, axis=-1)[:, : codes.shape[1]]


def _sigmoid(t):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(t, dtype=np.float64)))


_erfc = np.vectorize(math.erfc, otypes=[np.float64])
_P1 = math.sqrt(2.0 / math.pi)


def activation(z, kind) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if kind == "silu":
        return z * _sigmoid(z)
    if kind == "gelu":
        return z * _erfc(-z / math.sqrt(2.0)) / 2.0
    if kind == "gelu_tanh":
        return z * _sigmoid(2.0 * _P1 * (z + 0.044715 * z ** 3))
    return z


def activation_grad(z, kind) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if kind == "silu":
        s = _sigmoid(z)
        return s + z * s * _sigmoid(-z)
    if kind == "gelu":
        return _erfc(-z / math.sqrt(2.0)) / 2.0 + z * np.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = 2.0 * _P1 * (z + 0.044715 * z ** 3)
        return _sigmoid(t) + z * _sigmoid(t) * _sigmoid(-t) * 2.0 * _P1 * (1.0 + 3.0 * 0.044715 * z * z)
    return np.ones_like(z)


def silu_grads(grad_x, gate, up) -> tuple[np.ndarray, np.ndarray]:
    """float64 gradients of x = silu(gate) up."""
    gx, u = np.asarray(grad_x, dtype=np.float64), np.asarray(up, dtype=np.float64)
    return gx * u * activation_grad(gate, "silu"), gx * activation(gate, "silu")
