"""The linears return their output in the input's leading shape whatever shape of ``out`` the
caller gives it in.  On the host, with a library that records launches."""
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, nvfp4
from tests._fake_gpu import install, on_gpu

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 64, 32
BF = torch.bfloat16


@pytest.mark.parametrize("lead", [(M,), (2, M // 2), (1, M)])
@pytest.mark.parametrize("shape", [None, (M, N), (M * N,), (1, M * N), (M * N, 1), (2, M // 2, N)])
@pytest.mark.parametrize("name", ["linear", "swiglu", "segmented"])
def test_output_takes_the_inputs_shape(name, shape, lead, monkeypatch):
    install(monkeypatch, nvfp4)
    z = lambda *s, dtype=BF: on_gpu(torch.zeros(s, dtype=dtype))  # noqa: E731
    x = z(*lead, K)
    w = (z(N, K // 2, dtype=torch.uint8), z(nvfp4.scale_bytes(N, K), dtype=torch.uint8), on_gpu(torch.ones(())), None, N)
    ws = z(1 << 20, dtype=torch.uint8)
    out = z(M, N) if shape is None else z(*shape)
    call = {"linear": lambda: nvfp4.nvfp4_linear(x, *w, workspace=ws, out=out),
            "swiglu": lambda: nvfp4.nvfp4_linear_swiglu(x, x, *w, workspace=ws, out=out),
            "segmented": lambda: nvfp4.nvfp4_linear_segmented(x, 1, *w, workspace=ws, out=out)}[name]
    got = call()
    assert got.shape == (*lead, N) and got.data_ptr() == out.data_ptr()
