"""What a call writes into the caller's tensors counts as an in-place change for autograd, so a
gradient that saved one of them raises.  On the host, with a library that records launches."""
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, nvfp4
from tests._fake_gpu import install, on_gpu

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 64, 32
BF = torch.bfloat16


def z(*s, dtype=BF):
    return on_gpu(torch.zeros(s, dtype=dtype))


def test_versions(monkeypatch):
    install(monkeypatch, nvfp4)
    x, res, ws = z(M, K), z(M, N), z(1 << 20, dtype=torch.uint8)
    w = (z(N, K // 2, dtype=torch.uint8), z(nvfp4.scale_bytes(N, K), dtype=torch.uint8), on_gpu(torch.ones(())), None, N)
    codes, xs = z(M, K // 2, dtype=torch.uint8), z(nvfp4.scale_bytes(M, K), dtype=torch.uint8)
    g2 = on_gpu(torch.zeros(2))
    gemm = lambda **kw: nvfp4.nvfp4_gemm(codes, xs, w[0], w[1], w[2], w[2], workspace=ws, **kw)  # noqa: E731
    calls = [(lambda **kw: nvfp4.nvfp4_linear(x, *w, workspace=ws, **kw), True), (gemm, True),
             (lambda **kw: nvfp4.nvfp4_linear_swiglu(x, x, *w, workspace=ws, **kw), True),
             (lambda **kw: nvfp4.nvfp4_linear_segmented(x, 2, *w, workspace=ws, gsf_out=g2, **kw), False),
             (lambda **kw: nvfp4.nvfp4_linear_noalloc(x, *w, **kw), False)]
    for call, epilogue in calls:
        out, pre = z(M, N), z(M, N)
        before = out._version
        call(out=out)
        assert out._version > before
        if epilogue:
            before, pv = out._version, pre._version
            call(out=out, residual=res, preact=pre)
            assert out._version > before and pre._version > pv
    assert g2._version > 0 and res._version == x._version == ws._version == 0
    with torch.inference_mode():
        inner = on_gpu(torch.zeros((M, N), dtype=BF))
    gemm(out=inner)      # an inference tensor keeps no version: written as before


def test_a_saved_stream_raises(monkeypatch):
    install(monkeypatch, nvfp4)
    x, ws = z(M, K), z(1 << 20, dtype=torch.uint8)
    w = (z(N, K // 2, dtype=torch.uint8), z(nvfp4.scale_bytes(N, K), dtype=torch.uint8), on_gpu(torch.ones(())), None, N)
    a = torch.ones((M, N), dtype=BF, requires_grad=True)
    h = a * 2
    loss = (h * h).sum()                        # saves h
    nvfp4.nvfp4_linear(x, *w, workspace=ws, out=on_gpu(h.detach()), residual=on_gpu(h.detach()))
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
