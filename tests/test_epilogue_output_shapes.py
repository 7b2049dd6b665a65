"""An epilogue's out and preact take the shapes of the residual and of the plain linear's out:
rows of the output's width under any leading dimensions, or flat.  On the host, with a library
that records launches."""
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, nvfp4
from tests._fake_gpu import install, on_gpu

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 64, 32
BF = torch.bfloat16
GOOD = [(M, N), (2, M // 2, N), (1, M, N), (M * N,), (1, M * N)]


def z(*s, dtype=BF):
    return on_gpu(torch.zeros(s, dtype=dtype))


def _calls(lead):
    x = z(*lead, K)
    w = (z(N, K // 2, dtype=torch.uint8), z(nvfp4.scale_bytes(N, K), dtype=torch.uint8), on_gpu(torch.ones(())), None, N)
    ws = z(1 << 20, dtype=torch.uint8)
    codes, xs = z(M, K // 2, dtype=torch.uint8), z(nvfp4.scale_bytes(M, K), dtype=torch.uint8)
    return {"linear": lambda **kw: nvfp4.nvfp4_linear(x, *w, workspace=ws, **kw),
            "swiglu": lambda **kw: nvfp4.nvfp4_linear_swiglu(x, x, *w, workspace=ws, **kw),
            "gemm": lambda **kw: nvfp4.nvfp4_gemm(codes, xs, w[0], w[1], w[2], w[2], workspace=ws, **kw)}


@pytest.mark.parametrize("lead", [(M,), (2, M // 2)])
@pytest.mark.parametrize("shape", GOOD)
@pytest.mark.parametrize("name", ["linear", "swiglu", "gemm"])
def test_shapes(name, shape, lead, monkeypatch):
    rec = install(monkeypatch, nvfp4)
    call = _calls(lead)[name]
    out, pre = z(*shape), z(*shape)
    got = call(out=out, activation="silu", preact=pre)
    assert got.data_ptr() == out.data_ptr() and {out.data_ptr(), pre.data_ptr()} <= set(rec.calls[-1][1])
    assert got.shape == ((*lead, N) if name != "gemm" else shape)
    if shape[-1] == N:      # in place, as a residual of that shape
        assert call(out=out, residual=out).data_ptr() == out.data_ptr()
        assert rec.calls[-1][1].count(out.data_ptr()) == 2


@pytest.mark.parametrize("kw", [{"out": z(N, M)}, {"preact": z(N, M)}, {"out": z(M * N, 1)}, {"out": z(M, N + 1)},
                                {"preact": z(M * N - 1)}, {"preact": z(2, M * N)}])
@pytest.mark.parametrize("name", ["linear", "swiglu", "gemm"])
def test_other_shapes_are_refused(name, kw, monkeypatch):
    rec = install(monkeypatch, nvfp4)
    with pytest.raises(ValueError):
        _calls((M,))[name](activation="silu", **{"out": z(M, N), **kw})
    assert not rec.calls
