"""Outputs that a caller gives to the linears, on the GPU: refusals, and what lies behind a
larger buffer's part stays as it was."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _case(m, k, n):
    import nvfp4_w4a4_quantized_global_amd as nv
    x = workloads.draw("normal", (m, k), 230, m).to(DEV)
    return nv, x, nv.quantize_weight(workloads.draw("normal", (n, k), 231, n, 0.05).to(DEV))


@pytest.mark.parametrize("m", [1, 3, 20, 300])
def test_refused_without_an_epilogue(m):
    k, n = 256, 256
    nv, x, (pk, sc, gw) = _case(m, k, n)
    c, s, g = nv.quantize_activation(x)
    ref = nv.nvfp4_linear(x, pk, sc, gw, None, n)
    buf = torch.zeros((m + 1, n), dtype=BF, device=DEV)
    bad = (buf[:m - 1], buf.float()[:m], buf[:m].cpu(), torch.zeros((m, 2 * n), dtype=BF, device=DEV)[:, ::2], x)
    for out in bad:
        for call in (lambda: nv.nvfp4_linear(x, pk, sc, gw, None, n, out=out),
                     lambda: nv.nvfp4_linear_swiglu(x, x, pk, sc, gw, None, n, out=out),
                     lambda: nv.nvfp4_linear_segmented(x, 1, pk, sc, gw, None, n, out=out),
                     lambda: nv.nvfp4_linear_noalloc(x, pk, sc, gw, None, n, out=out)):
            with pytest.raises(ValueError):
                call()
        if out is not x:      # the product reads the codes
            with pytest.raises(ValueError):
                nv.nvfp4_gemm(c, s, pk, sc, g, gw, out=out)
    with pytest.raises(ValueError):
        nv.nvfp4_linear(x, pk, sc, gw, None, n, workspace=torch.zeros(1 << 24, dtype=torch.uint8))
    assert torch.equal(nv.nvfp4_linear(x, pk, sc, gw, None, n), ref)      # nothing is left behind
    buf[m:] = 7.0
    got = nv.nvfp4_gemm(c, s, pk, sc, g, gw, out=buf)
    assert got is buf and torch.equal(buf[:m], nv.nvfp4_gemm(c, s, pk, sc, g, gw)) and bool((buf[m:] == 7.0).all())
