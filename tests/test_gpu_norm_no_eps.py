"""The RMS norm's gradient without an eps, on row counts that leave a workgroup partly empty:
the rows that are not there contribute nothing to grad_w."""
import numpy as np
import pytest
import torch

import oracle as o
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def _f(t):
    return t.detach().float().cpu().numpy()


# rows of at most 1024 values share a workgroup: 32 of 128 values, 4 of 1024
@pytest.mark.parametrize("m,k", [(1, 16), (1, 128), (31, 128), (33, 64), (5, 1024), (4097, 512), (3, 1040), (4, 1024)])
@pytest.mark.parametrize("rd", [torch.bfloat16, torch.float32])
def test_rows_that_are_not_there(m, k, rd):
    import nvfp4_w4a4_quantized_global_amd as nv
    r = workloads.draw("normal", (m, k), 220, 0).to(rd)
    w = 1.0 + 0.1 * workloads.draw("normal", (k,), 221, 1).float()
    gy = workloads.draw("normal", (m, k), 222, 2, 1e-2)
    gx, gw = nv.rmsnorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), 0.0)
    ref_x, ref_w = o.rmsnorm_grads(_f(gy), _f(r), _f(w), 0.0)
    # a term gy r s carries three roundings, its sum over the rows one an addition
    g, n = np.abs(_f(gy).astype(np.float64)), np.abs(_f(r)) / np.sqrt(np.mean(_f(r).astype(np.float64) ** 2, -1, keepdims=True))
    assert np.all(np.abs(_f(gw) - ref_w) <= U * (m + 4) * np.sum(g * n, 0))
    # s g and n f take at most eight roundings, d = sum(g r) fifty on the way of a term
    s = 1.0 / np.sqrt(np.mean(_f(r).astype(np.float64) ** 2, -1, keepdims=True))
    gv = g * np.abs(_f(w))
    tol = U * (8 * s * gv + 50 * n * s * np.mean(gv * n, -1, keepdims=True))
    if rd == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref_x) + tol)
    assert np.all(np.abs(_f(gx) - ref_x) <= tol + 2.0 ** -134)


@pytest.mark.parametrize("m,k", [(1, 48), (1, 512), (5, 144), (33, 64), (3, 1040)])
def test_forward_forms(m, k):
    """The codes of every form without an eps equal those of the written norm."""
    import nvfp4_w4a4_quantized_global_amd as nv
    x = workloads.draw("normal", (m, k), 223, 0).to(DEV)
    w = (1.0 + 0.1 * workloads.draw("normal", (k,), 224, 1).float()).to(DEV)
    y = nv.rmsnorm(x, w, 0.0)
    assert np.array_equal(_f(y), o.rmsnorm(_f(x), _f(w), 0.0)[1])
    for gsf in (None, 4.0):
        got, ref = nv.quantize_rmsnorm(x, w, 0.0, None, gsf), nv.quantize_activation(y, gsf)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    ck, ref = nv.rmsnorm_checkpoint(x, w, 0.0)[1], nv.checkpoint_pack(y)
    assert torch.equal(ck.codes, ref.codes) and torch.equal(ck.scales, ref.scales)
