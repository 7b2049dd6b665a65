"""Outputs and workspaces that a caller gives to the linears: what a kernel would write past,
or on the wrong device, or into rows that it still reads, is refused before anything is
launched.  On the host, with a library that records launches."""
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, nvfp4
from tests._fake_gpu import install, on_gpu

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 64, 32
BF = torch.bfloat16


def _z(*shape, dtype=BF):
    return on_gpu(torch.zeros(shape, dtype=dtype))


def _calls():
    """name -> (call(out, workspace), the activation it reads)."""
    x = _z(M, K)
    packed, scales = _z(N, K // 2, dtype=torch.uint8), _z(nvfp4.scale_bytes(N, K), dtype=torch.uint8)
    codes = _z(4096, dtype=torch.uint8)[:M * K // 2].view(M, K // 2)     # with room behind them
    xs = _z(nvfp4.scale_bytes(M, K), dtype=torch.uint8)
    g = on_gpu(torch.ones(()))
    up, res = _z(M, K), _z(M, N)
    w = (packed, scales, g, None, N)
    return {
        "linear": (lambda o, ws: nvfp4.nvfp4_linear(x, *w, workspace=ws, out=o), x),
        "linear_epilogue": (lambda o, ws: nvfp4.nvfp4_linear(x, *w, workspace=ws, out=o, residual=res), x),
        "gemm": (lambda o, ws: nvfp4.nvfp4_gemm(codes, xs, packed, scales, g, g, out=o, workspace=ws), codes),
        "gemm_epilogue": (lambda o, ws: nvfp4.nvfp4_gemm(codes, xs, packed, scales, g, g, out=o, workspace=ws,
                                                         activation="gelu"), codes),
        "swiglu": (lambda o, ws: nvfp4.nvfp4_linear_swiglu(x, up, *w, workspace=ws, out=o), up),
        "swiglu_epilogue": (lambda o, ws: nvfp4.nvfp4_linear_swiglu(x, up, *w, workspace=ws, out=o, residual=res), up),
        "segmented": (lambda o, ws: nvfp4.nvfp4_linear_segmented(x, 2, *w, workspace=ws, out=o), x),
        "noalloc": (lambda o, ws: nvfp4.nvfp4_linear_noalloc(x, *w, out=o), x),
    }


NAMES = ["linear", "linear_epilogue", "gemm", "gemm_epilogue", "swiglu", "swiglu_epilogue", "segmented", "noalloc"]


def _workspace():
    return _z(1 << 20, dtype=torch.uint8)


@pytest.mark.parametrize("name", NAMES)
def test_bad_outputs_are_refused(name, monkeypatch):
    rec = install(monkeypatch, nvfp4)
    call, x = _calls()[name]
    bad = {"short": _z(M - 1, N), "empty": _z(0, N), "on the host": torch.zeros((M, N), dtype=BF), "fp32": _z(M, N, dtype=torch.float32),
           "fp16": _z(M, N, dtype=torch.float16), "strided": on_gpu(torch.zeros((M, 2 * N), dtype=BF)[:, ::2]),
           "another device": on_gpu(torch.zeros((M, N), dtype=BF), 1)}
    if name != "gemm":
        bad["long"] = _z(M + 1, N)
    for what, out in bad.items():
        with pytest.raises(ValueError):
            call(out, _workspace())
        assert not rec.calls, what


@pytest.mark.parametrize("name", NAMES)
def test_an_output_over_the_input_is_refused(name, monkeypatch):
    rec = install(monkeypatch, nvfp4)
    call, x = _calls()[name]
    values = x.numel() * x.element_size() // 2       # bf16 values; the output ends with the input, or begins with it
    first = max(values - M * N, 0)
    out = torch.as_strided(x.view(BF), (M, N), (N, 1), first)
    with pytest.raises(ValueError):
        call(on_gpu(out), _workspace())
    assert not rec.calls


@pytest.mark.parametrize("name", NAMES)
def test_good_outputs_are_written(name, monkeypatch):
    rec = install(monkeypatch, nvfp4)
    call, _ = _calls()[name]
    out = _z(M, N)
    got = call(out, _workspace())
    assert len(rec.calls) == 1 and out.data_ptr() in rec.calls[0][1]
    assert got.data_ptr() == out.data_ptr() and got.shape == (M, N)


@pytest.mark.parametrize("name", ["linear", "gemm", "swiglu", "segmented"])
def test_flat_outputs_without_an_epilogue(name, monkeypatch):
    """As many values in another shape, and for the bare product room for more."""
    rec = install(monkeypatch, nvfp4)
    call, _ = _calls()[name]
    outs = [_z(M * N), _z(2, M // 2, N)] + ([_z(M + 3, N)] if name == "gemm" else [])
    for out in outs:
        assert call(out, _workspace()).data_ptr() == out.data_ptr()
    assert len(rec.calls) == len(outs)


@pytest.mark.parametrize("name", [n for n in NAMES if n != "noalloc"])
def test_bad_workspaces_are_refused(name, monkeypatch):
    rec = install(monkeypatch, nvfp4)
    call, _ = _calls()[name]
    host, other = torch.zeros(1 << 20, dtype=torch.uint8), on_gpu(torch.zeros(1 << 20, dtype=torch.uint8), 1)
    one = on_gpu(torch.zeros(1, dtype=torch.uint8).expand(1 << 20))       # a byte, a million times
    for ws in (host, other, one):
        with pytest.raises(ValueError):
            call(_z(M, N), ws)
    assert not rec.calls
