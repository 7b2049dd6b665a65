"""Refusals of the norm, epilogue and checkpoint calls at the C ABI, before anything is
queued: these run without a GPU."""
import ctypes
import os

import pytest

from nvfp4_w4a4_quantized_global_amd import _lib
from nvfp4_w4a4_quantized_global_amd._lib import NVFP4_ERR_ARG, NVFP4_ERR_SHAPE, NVFP4_ERR_WORKSPACE, lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
P = ctypes.c_void_p(0x1000)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1008)
ODD1 = ctypes.c_void_p(0x1001)


def _msg():
    return lib().nvfp4_last_error().decode()


def _norm(rows=4, k=64, xd=0, res=None, rd=0, wd=0, eps=1e-6, x=P, w=P, r=P, y=P, cc=None, cs=None):
    return lib().nvfp4_rmsnorm(x, xd, res, rd, w, wd, rows, k, eps, r, y, cc, cs, None)


def test_norm_refusals():
    for k in (0, 8, 24, 16400, -16):
        assert _norm(k=k) == NVFP4_ERR_SHAPE
    assert "16384" in (_norm(k=16400), _msg())[1]
    assert _norm(rows=-1) == NVFP4_ERR_SHAPE and _norm(rows=1 << 31) == NVFP4_ERR_SHAPE
    for bad in ({"xd": 2}, {"wd": -1}, {"res": P, "rd": 7}, {"xd": 1, "res": P, "rd": 0}, {"eps": -1.0},
                {"eps": float("nan")}, {"eps": float("inf")}, {"x": None}, {"w": None}, {"y": None},
                {"res": P, "r": None}, {"x": ODD}, {"w": ODD}, {"y": ODD}, {"res": ODD}, {"res": P, "r": ODD},
                {"cc": P}, {"cs": P}, {"cc": ODD, "cs": P}):
        assert _norm(**bad) == NVFP4_ERR_ARG, bad
    assert _norm(rows=0, x=None, w=None, y=None) == 0


def test_quantize_norm_refusals():
    def q(gsf=None, codes=P, scales=P, ws=P, n=1 << 20, rows=4, g=None):
        return lib().nvfp4_quantize_rmsnorm(P, 0, None, 0, P, 0, rows, 64, 1e-6, gsf, None, codes, scales, g, ws, n, None)

    need = lib().nvfp4_quantize_rmsnorm_workspace_bytes(4)
    assert need % 256 == 0 and need >= 4 * 4
    assert lib().nvfp4_quantize_rmsnorm_workspace_bytes(-1) == 0
    assert q(codes=None) == NVFP4_ERR_ARG and q(scales=None) == NVFP4_ERR_ARG
    assert q(codes=ctypes.c_void_p(0x1004)) == NVFP4_ERR_ARG and q(gsf=ctypes.c_void_p(0x1002)) == NVFP4_ERR_ARG
    assert q(g=ODD1) == NVFP4_ERR_ARG
    assert q(ws=None) == NVFP4_ERR_WORKSPACE and q(n=need - 1) == NVFP4_ERR_WORKSPACE and q(ws=ODD) == NVFP4_ERR_WORKSPACE
    assert q(rows=0, codes=None, scales=None, ws=None) == 0


def test_norm_backward_refusals():
    def b(gy=P, r=P, rd=0, w=P, wd=0, gres=None, rows=4, k=64, gr=P, gw=P, ws=P, n=1 << 20):
        return lib().nvfp4_rmsnorm_backward(gy, r, rd, w, wd, gres, rows, k, 1e-6, gr, gw, ws, n, None)

    assert b(k=24) == NVFP4_ERR_SHAPE and b(k=16400) == NVFP4_ERR_SHAPE
    for bad in ({"rd": 3}, {"wd": 3}, {"gy": None}, {"r": None}, {"w": None}, {"gr": None}, {"gy": ODD}, {"gres": ODD},
                {"gr": ODD}, {"gw": ODD1}):
        assert b(**bad) == NVFP4_ERR_ARG, bad
    assert b(ws=None) == NVFP4_ERR_WORKSPACE
    assert b(n=lib().nvfp4_rmsnorm_backward_workspace_bytes(4, 64) - 1) == NVFP4_ERR_WORKSPACE
    assert lib().nvfp4_rmsnorm_backward_workspace_bytes(4, 24) == 0
    assert b(rows=0, gw=None, ws=None) == 0


def test_checkpoint_refusals():
    L = lib()
    assert L.nvfp4_checkpoint_scale_bytes(3, 48) == 6 and L.nvfp4_checkpoint_scale_bytes(0, 64) == 0
    assert L.nvfp4_checkpoint_pack(P, 4, 24, 0, P, P, None) == NVFP4_ERR_SHAPE
    assert L.nvfp4_checkpoint_pack(P, 4, 64, 3, P, P, None) == NVFP4_ERR_ARG
    assert L.nvfp4_checkpoint_pack(P, 4, 48, 32, P, P, None) == NVFP4_ERR_ARG and "does not divide" in _msg()
    for a in ((None, P, P), (P, None, P), (P, P, None), (ODD, P, P), (P, ODD, P)):
        assert L.nvfp4_checkpoint_pack(a[0], 4, 64, 0, a[1], a[2], None) == NVFP4_ERR_ARG
        assert L.nvfp4_checkpoint_unpack(a[1], a[2], 4, 64, a[0], 0, None) == NVFP4_ERR_ARG
    assert L.nvfp4_checkpoint_unpack(P, P, 4, 64, P, 2, None) == NVFP4_ERR_ARG
    assert L.nvfp4_swiglu_checkpoint(P, P, 4, 64, P, P, None, P, P, None) == NVFP4_ERR_ARG
    assert L.nvfp4_swiglu_checkpoint(P, ODD, 4, 64, P, P, P, P, P, None) == NVFP4_ERR_ARG
    assert L.nvfp4_swiglu_backward(P, P, P, P, None, 4, 64, P, P, None) == NVFP4_ERR_ARG and "both" in _msg()
    assert L.nvfp4_swiglu_backward(P, P, None, P, None, 4, 24, P, P, None) == NVFP4_ERR_SHAPE
    assert L.nvfp4_swiglu_backward(ODD, P, None, P, None, 4, 64, P, P, None) == NVFP4_ERR_ARG
    assert L.nvfp4_activation_backward(P, P, None, 4, 24, 9, P, None) == NVFP4_ERR_ARG
    assert L.nvfp4_activation_backward(P, P, P, 4, 24, 1, P, None) == NVFP4_ERR_SHAPE     # a checkpoint: n % 16
    assert L.nvfp4_activation_backward(P, P, None, 4, 0, 1, P, None) == NVFP4_ERR_SHAPE
    assert L.nvfp4_activation_backward(P, None, None, 4, 24, 1, P, None) == NVFP4_ERR_ARG


def test_weight_grad_refusals():
    L = lib()

    def w(gy=P, m=4, n=8, c=P, s=P, k=64, out=P, d=1, ws=None, b=0):
        return L.nvfp4_weight_grad(gy, m, n, c, s, k, out, d, ws, b, None)

    assert w(k=24) == NVFP4_ERR_SHAPE and w(n=0) == NVFP4_ERR_SHAPE and w(m=-1) == NVFP4_ERR_SHAPE
    for bad in ({"gy": None}, {"c": None}, {"s": None}, {"out": None}, {"gy": ODD}, {"c": ODD}, {"out": ODD}, {"d": 2}):
        assert w(**bad) == NVFP4_ERR_ARG, bad
    assert w(ws=ODD, b=1 << 20) == NVFP4_ERR_WORKSPACE
    assert L.nvfp4_weight_grad_workspace_bytes(-1, 8, 64) == 0


def test_epilogue_refusals():
    L = lib()
    need = L.nvfp4_linear_workspace_bytes(4, 64, 8)
    ws = ctypes.c_void_p(0x10000)

    def e(act=1, res=None, pre=None, up=None, g=0, out=P, n=need):
        return L.nvfp4_linear_epilogue(P, up, 4, 64, P, P, P, None, 8, None, g, act, res, pre, out, ws, n, None)

    for bad in ({"act": 4}, {"act": -1}, {"res": ODD1}, {"pre": ODD1}, {"pre": P}, {"res": ODD, "pre": ODD},
                {"up": P, "g": 16}, {"up": ODD}):
        assert e(**bad) == NVFP4_ERR_ARG, bad
    assert e(n=need - 1) == NVFP4_ERR_WORKSPACE
    assert e(up=P) == NVFP4_ERR_WORKSPACE            # the SwiGLU product needs more
    assert L.nvfp4_gemm_epilogue(P, P, 4, 64, P, P, 8, P, P, None, 5, None, None, P, None, 0, None) == NVFP4_ERR_ARG
    assert L.nvfp4_gemm_epilogue(P, P, 4, 24, P, P, 8, P, P, None, 1, None, None, P, None, 0, None) == NVFP4_ERR_SHAPE
    assert L.nvfp4_linear_epilogue(None, None, 0, 64, None, None, None, None, 8, None, 0, 1, None, None, None, None, 0,
                                   None) == 0
