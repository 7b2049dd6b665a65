"""Plain definitions of the layer norm with its gradient and of the 8-bit block format with its
product.

Real-valued steps are float64; where the contract fixes a rounding (the norm's centred value,
scale and output, the format's scale and factor) it is applied explicitly.  Pins:
tests/test_oracle_blocks.py.
"""
from __future__ import annotations

import numpy as np

from .nvfp4 import bf16_round, e4m3_decode

__all__ = ["layernorm", "layernorm_grads", "fp8_quantize", "fp8_values", "FP8_FLOOR"]

BLOCK = 128
FP8_FLOOR = 448.0 * 2.0 ** -110


def _f32(a):
    return np.asarray(a, dtype=np.float64).astype(np.float32)


def layernorm(x, weight, bias, eps, residual=None, stream: str = "bf16") -> tuple[np.ndarray, np.ndarray]:
    """(r, y): r = x + residual in fp32, rounded to the stream's type; y =
    bf16(fp32(fp32(fp32(r - mu) * s) * w) + b), mu and the variance in float64 and
    s = fp32(1 / sqrt(variance + eps))."""
    r = _f32(x)
    if residual is not None:
        r = (r + _f32(residual)).astype(np.float32)
        if stream == "bf16":
            r = bf16_round(r)
    d = r.astype(np.float64)
    c = d - np.mean(d, axis=-1, keepdims=True)
    s = _f32(1.0 / np.sqrt(np.mean(c * c, axis=-1, keepdims=True) + np.float64(np.float32(eps))))
    y = ((_f32(c) * s).astype(np.float32) * _f32(weight)).astype(np.float32)
    if bias is not None:
        y = (y + _f32(bias)).astype(np.float32)
    return r, bf16_round(y)


def layernorm_grads(grad_y, r, weight, eps, grad_residual=None) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """float64 gradients of y = (r - mu) / sqrt(var + eps) w + b for r, w and b."""
    r, gy, w = (np.asarray(a, dtype=np.float64) for a in (r, grad_y, weight))
    c = r - np.mean(r, axis=-1, keepdims=True)
    s = 1.0 / np.sqrt(np.mean(c * c, axis=-1, keepdims=True) + np.float64(np.float32(eps)))
    n, g = c * s, gy * w
    grad_r = s * (g - np.mean(g, axis=-1, keepdims=True) - n * np.mean(g * n, axis=-1, keepdims=True))
    if grad_residual is not None:
        grad_r = grad_r + np.asarray(grad_residual, dtype=np.float64)
    return grad_r, np.sum(gy * n, axis=0), np.sum(gy, axis=0)


def _per_value(a, rows: int, shape) -> np.ndarray:
    """[tiles down, tiles across] spread over a matrix of ``shape``, tiles of rows x 128."""
    return np.repeat(np.repeat(a, rows, axis=0)[: shape[0]], BLOCK, axis=1)[:, : shape[1]]


def fp8_quantize(x, rows: int) -> tuple[np.ndarray, np.ndarray]:
    """uint8 E4M3 codes [M, K] and fp32 scales [ceil(M/rows), ceil(K/128)] of tiles of rows x 128
    (rows 1: an activation, before its scales are transposed; 128: a weight): the nearest E4M3 value
    to fp32(v fp32(448 / a)), by search, ties to the even code; NaN for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    m, k = x.shape
    fine = np.isfinite(x)
    a = np.zeros((-(-m // rows), -(-k // BLOCK)))
    for i in range(a.shape[0]):
        for j in range(a.shape[1]):
            t = np.s_[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
            a[i, j] = np.max(np.where(fine[t], np.abs(x[t]), 0.0))
    a = np.maximum(a, FP8_FLOOR)
    factor = _per_value(_f32(448.0 / a), rows, x.shape).astype(np.float64)
    v = _f32(np.where(fine, x, 0.0) * factor).astype(np.float64)
    grid = e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, np.abs(v), side="left"), np.searchsorted(mid, np.abs(v), side="right")
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo).astype(np.uint8)
    code = np.where(fine, code | (np.signbit(x).astype(np.uint8) << 7), np.uint8(0x7F))
    return code, _f32(a / 448.0)


def fp8_values(codes, scales, rows: int) -> np.ndarray:
    """float64 code * scale (NaN codes as NaN)."""
    codes = np.asarray(codes, dtype=np.uint8)
    mag = codes & 0x7F
    v = np.where(mag == 0x7F, np.nan, e4m3_decode(np.minimum(mag, 126)).astype(np.float64))
    return np.where(codes & 0x80, -v, v) * _per_value(np.asarray(scales, dtype=np.float64), rows, codes.shape)
