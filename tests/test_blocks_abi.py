"""Refusals of the layer norm and 8-bit block calls at the C ABI, before anything is queued: these
run without a GPU."""
import ctypes
import os

import pytest

from nvfp4_w4a4_quantized_global_amd import _lib
from nvfp4_w4a4_quantized_global_amd._lib import NVFP4_ERR_ARG, NVFP4_ERR_SHAPE, NVFP4_ERR_WORKSPACE, lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
P = ctypes.c_void_p(0x1000)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1008)
ODD1 = ctypes.c_void_p(0x1001)
MAX = 1 << 22


def _msg():
    return lib().nvfp4_last_error().decode()


def test_layernorm_refusals():
    def n(rows=4, k=64, xd=0, res=None, rd=0, w=P, b=None, wd=0, eps=1e-6, x=P, r=P, y=P, cc=None, cs=None):
        return lib().nvfp4_layernorm(x, xd, res, rd, w, b, wd, rows, k, eps, r, y, cc, cs, None)

    for k in (0, 8, 24, 16400, -16):
        assert n(k=k) == NVFP4_ERR_SHAPE
    assert "16384" in (n(k=16400), _msg())[1]
    assert n(rows=-1) == NVFP4_ERR_SHAPE and n(rows=1 << 31) == NVFP4_ERR_SHAPE
    for bad in ({"xd": 2}, {"wd": -1}, {"res": P, "rd": 7}, {"xd": 1, "res": P, "rd": 0}, {"eps": -1.0},
                {"eps": float("nan")}, {"eps": float("inf")}, {"x": None}, {"w": None}, {"y": None}, {"b": ODD},
                {"res": P, "r": None}, {"x": ODD}, {"w": ODD}, {"y": ODD}, {"res": ODD}, {"res": P, "r": ODD},
                {"cc": P}, {"cs": P}, {"cc": ODD, "cs": P}):
        assert n(**bad) == NVFP4_ERR_ARG, bad
    assert n(rows=0, x=None, w=None, y=None) == 0


def test_quantize_layernorm_refusals():
    def q(gsf=None, codes=P, scales=P, ws=P, n=1 << 20, rows=4, g=None, b=None):
        return lib().nvfp4_quantize_layernorm(P, 0, None, 0, P, b, 0, rows, 64, 1e-6, gsf, None, codes, scales, g, ws, n, None)

    need = lib().nvfp4_quantize_layernorm_workspace_bytes(4)
    assert need % 256 == 0 and need >= 4 * 12
    assert lib().nvfp4_quantize_layernorm_workspace_bytes(-1) == 0 == lib().nvfp4_quantize_layernorm_workspace_bytes(1)
    assert q(codes=None) == NVFP4_ERR_ARG and q(scales=None) == NVFP4_ERR_ARG and q(b=ODD) == NVFP4_ERR_ARG
    assert q(codes=ctypes.c_void_p(0x1004)) == NVFP4_ERR_ARG and q(gsf=ctypes.c_void_p(0x1002)) == NVFP4_ERR_ARG
    assert q(g=ODD1) == NVFP4_ERR_ARG
    assert q(ws=None) == NVFP4_ERR_WORKSPACE and q(n=need - 1) == NVFP4_ERR_WORKSPACE and q(ws=ODD) == NVFP4_ERR_WORKSPACE
    assert q(rows=0, codes=None, scales=None, ws=None) == 0


def test_layernorm_backward_refusals():
    def b(gy=P, r=P, rd=0, w=P, wd=0, gres=None, rows=4, k=64, gr=P, gw=P, gb=P, ws=P, n=1 << 20):
        return lib().nvfp4_layernorm_backward(gy, r, rd, w, wd, gres, rows, k, 1e-6, gr, gw, gb, ws, n, None)

    assert b(k=24) == NVFP4_ERR_SHAPE and b(k=16400) == NVFP4_ERR_SHAPE
    for bad in ({"rd": 3}, {"wd": 3}, {"gy": None}, {"r": None}, {"w": None}, {"gr": None}, {"gy": ODD}, {"gres": ODD},
                {"gr": ODD}, {"gw": ODD1}, {"gb": ODD1}, {"gw": None}, {"gb": None}):
        assert b(**bad) == NVFP4_ERR_ARG, bad
    need = lib().nvfp4_layernorm_backward_workspace_bytes(4, 64)
    assert b(ws=None) == NVFP4_ERR_WORKSPACE and b(n=need - 1) == NVFP4_ERR_WORKSPACE
    assert lib().nvfp4_layernorm_backward_workspace_bytes(4, 24) == 0
    assert b(rows=0, gw=None, gb=None, ws=None) == 0


def test_fp8_quantize_refusals():
    L = lib()

    def a(x=P, up=None, rows=4, k=64, c=P, s=P, t=None, ws=None, n=0):
        return L.nvfp4_fp8_quantize_activation(x, up, rows, k, c, s, t, ws, n, None)

    for k in (0, 8, 24, MAX + 16):
        assert a(k=k) == NVFP4_ERR_SHAPE
    assert a(rows=-1) == NVFP4_ERR_SHAPE
    for bad in ({"x": None}, {"c": None}, {"s": None}, {"x": ODD}, {"up": ODD}, {"c": ODD}, {"s": ODD1}, {"up": P, "t": P},
                {"t": ODD1, "ws": P, "n": 1 << 20}):
        assert a(**bad) == NVFP4_ERR_ARG, bad
    need = L.nvfp4_fp8_quantize_workspace_bytes(4, 64)
    assert need >= 256 and L.nvfp4_fp8_quantize_workspace_bytes(-1, 64) == 0
    assert a(t=P) == NVFP4_ERR_WORKSPACE and a(t=P, ws=P, n=need - 1) == NVFP4_ERR_WORKSPACE
    assert a(rows=0, x=None, c=None, s=None) == 0

    def q(x=P, rows=4, k=64, c=P, s=P, kc=P, ks=P):
        return L.nvfp4_fp8_quantize_checkpoint(x, rows, k, c, s, kc, ks, None)

    for bad in ({"k": 24}, {"k": MAX + 16}, {"rows": -1}):
        assert q(**bad) == NVFP4_ERR_SHAPE, bad
    for bad in ({"x": None}, {"c": None}, {"s": None}, {"kc": None}, {"ks": None}, {"x": ODD}, {"c": ODD}, {"s": ODD1}, {"kc": ODD}):
        assert q(**bad) == NVFP4_ERR_ARG, bad
    assert q(rows=0, x=None, c=None, s=None, kc=None, ks=None) == 0

    def w(x=P, d=0, n=32, k=64, c=P, s=P, ct=None, st=None):
        return L.nvfp4_fp8_quantize_weight(x, d, n, k, c, s, ct, st, None)

    assert w(k=24) == NVFP4_ERR_SHAPE and w(n=0) == NVFP4_ERR_SHAPE and w(n=MAX + 1) == NVFP4_ERR_SHAPE
    assert w(n=20, ct=P, st=P) == NVFP4_ERR_SHAPE and "divisible" in _msg()
    for bad in ({"d": 2}, {"x": None}, {"c": None}, {"s": None}, {"x": ODD}, {"c": ODD}, {"s": ODD1}, {"ct": P}, {"st": P},
                {"ct": ODD, "st": P}, {"ct": P, "st": ODD1}):
        assert w(**bad) == NVFP4_ERR_ARG, bad

    def d(c=P, s=P, rows=4, k=64, wt=0, o=P, od=0):
        return L.nvfp4_fp8_dequantize(c, s, rows, k, wt, o, od, None)

    assert d(k=24) == NVFP4_ERR_SHAPE
    for bad in ({"od": 2}, {"c": None}, {"s": None}, {"o": None}, {"c": ODD}, {"s": ODD1}, {"o": ODD}):
        assert d(**bad) == NVFP4_ERR_ARG, bad
    assert d(rows=0, c=None, s=None, o=None) == 0


@pytest.mark.parametrize("layer", [True, False])
def test_fp8_quantize_norm_refusals(layer):
    def q(rows=4, k=64, xd=0, res=None, rd=0, w=P, b=None, x=P, r=P, c=P, s=P):
        if layer:
            return lib().nvfp4_fp8_quantize_layernorm(x, xd, res, rd, w, b, 0, rows, k, 1e-6, r, c, s, None)
        return lib().nvfp4_fp8_quantize_rmsnorm(x, xd, res, rd, w, 0, rows, k, 1e-6, r, c, s, None)

    assert q(k=24) == NVFP4_ERR_SHAPE and q(k=16400) == NVFP4_ERR_SHAPE and q(rows=-1) == NVFP4_ERR_SHAPE
    for bad in ({"xd": 2}, {"x": None}, {"w": None}, {"c": None}, {"s": None}, {"c": ODD}, {"s": ODD1}, {"x": ODD},
                {"res": P, "r": None}, {"xd": 1, "res": P}):
        assert q(**bad) == NVFP4_ERR_ARG, bad
    if layer:
        assert q(b=ODD) == NVFP4_ERR_ARG
    assert q(rows=0, x=None, w=None, c=None, s=None) == 0


def test_fp8_product_refusals():
    L = lib()

    def g(xc=P, xs=P, m=4, k=64, wc=P, ws=P, n=32, b=None, act=0, res=None, pre=None, o=P, wk=None, nb=0):
        return L.nvfp4_fp8_gemm(xc, xs, m, k, wc, ws, n, b, act, res, pre, o, wk, nb, None)

    def li(x=P, up=None, m=4, k=64, wc=P, ws=P, b=None, n=32, act=0, res=None, pre=None, o=P, wk=P, nb=1 << 30):
        return L.nvfp4_fp8_linear(x, up, m, k, wc, ws, b, n, act, res, pre, o, wk, nb, None)

    for f in (g, li):
        assert f(k=24) == NVFP4_ERR_SHAPE and f(k=MAX + 16) == NVFP4_ERR_SHAPE and f(m=-1) == NVFP4_ERR_SHAPE
        assert f(n=0) == NVFP4_ERR_SHAPE and f(n=MAX + 1) == NVFP4_ERR_SHAPE
        for bad in ({"wc": None}, {"ws": None}, {"o": None}, {"wc": ODD}, {"ws": ODD1}, {"o": ODD1}, {"b": ODD1}, {"act": 4},
                    {"act": -1}, {"res": ODD1}, {"pre": ODD1}, {"pre": P}, {"res": P, "pre": P, "o": ODD}):
            assert f(**bad) == NVFP4_ERR_ARG, bad
        assert f(m=0, wc=None, ws=None, o=None) == 0
    for bad in ({"xc": None}, {"xs": None}, {"xc": ODD}, {"xs": ODD1}):
        assert g(**bad) == NVFP4_ERR_ARG, bad
    assert g(m=300, wk=ODD, nb=1 << 30) == NVFP4_ERR_WORKSPACE
    for bad in ({"x": None}, {"x": ODD}, {"up": ODD}):
        assert li(**bad) == NVFP4_ERR_ARG, bad
    need = L.nvfp4_fp8_linear_workspace_bytes(300, 64, 32)
    assert li(m=300, wk=None) == NVFP4_ERR_WORKSPACE and li(m=300, nb=need - 1) == NVFP4_ERR_WORKSPACE
    assert li(m=300, wk=ODD) == NVFP4_ERR_WORKSPACE


def test_fp8_sizes():
    L = lib()
    # one to four rows quantize inside the product while their codes fit a workgroup's LDS
    assert L.nvfp4_fp8_linear_workspace_bytes(1, 5120, 1024) == 0 == L.nvfp4_fp8_linear_workspace_bytes(4, 5120, 1024)
    assert L.nvfp4_fp8_linear_workspace_bytes(4, 25600, 1024) > 4 * 25600
    # else codes and scales, and the split products' partials
    assert L.nvfp4_fp8_linear_workspace_bytes(16, 5120, 1024) == 16 * 5120 + 40 * 16 * 4
    assert L.nvfp4_fp8_linear_workspace_bytes(300, 5120, 1024) == \
        300 * 5120 + (40 * 300 * 4 + 255) // 256 * 256 + L.nvfp4_fp8_gemm_workspace_bytes(300, 5120, 1024)
    # 24 tiles of 128 x 128 split along K: whole fp32 tiles of each part
    part = L.nvfp4_fp8_gemm_workspace_bytes(300, 5120, 1024)
    assert part > 0 and part % (24 * 128 * 128 * 4) == 0
    assert L.nvfp4_fp8_gemm_workspace_bytes(4096, 5120, 16384) == 0          # whole rounds
    assert L.nvfp4_fp8_gemm_workspace_bytes(1, 5120, 1024) == 0 == L.nvfp4_fp8_gemm_workspace_bytes(0, 64, 64)
    # partials never exceed one round of tiles: 256 of 256 x 256, or 512 of 128 x 128
    for m, k, n in ((33, 1 << 20, 16), (4096, 25600, 5120), (100, 8192, 8192), (1000, 16, 1000)):
        assert L.nvfp4_fp8_gemm_workspace_bytes(m, k, n) <= 256 * 256 * 256 * 4


def test_sizes_outside_the_calls_limits():
    L = lib()
    most, wide = (1 << 31) - 1, 1 << 22
    assert L.nvfp4_fp8_linear_workspace_bytes(most, wide, wide) > most * wide
    assert L.nvfp4_layernorm_backward_workspace_bytes(most, 16384) > 0 < L.nvfp4_quantize_layernorm_workspace_bytes(most)
    assert L.nvfp4_fp8_quantize_workspace_bytes(most, wide) > 0
    for big in (1 << 31, (1 << 63) - 1, -1):
        assert L.nvfp4_layernorm_backward_workspace_bytes(big, 5120) == 0 == L.nvfp4_quantize_layernorm_workspace_bytes(big)
        assert L.nvfp4_fp8_quantize_workspace_bytes(big, 5120) == 0 == L.nvfp4_fp8_quantize_workspace_bytes(16, big)
        for f in (L.nvfp4_fp8_gemm_workspace_bytes, L.nvfp4_fp8_linear_workspace_bytes):
            assert f(big, 512, 512) == 0 == f(300, big, 512) == f(300, 512, big)
