"""The residual's gradient of the training linear is a tensor of its own: accumulating into it
over several backward passes leaves the caller's gradient, and the other leaves', alone."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("kw", [{}, {"checkpoint": True}, {"activation": "gelu"}, {"checkpoint": True, "activation": "silu"}])
@pytest.mark.parametrize("shape", [(4, 48), (2, 2, 48), (1, 4, 48)])
def test_accumulates_alone(shape, kw):
    import nvfp4_w4a4_quantized_global_amd as nv
    x = workloads.draw("normal", (4, 64), 240, 0).to(DEV)
    w = workloads.draw("normal", (48, 64), 240, 1).to(DEV)
    gy = workloads.draw("normal", (4, 48), 240, 2).to(DEV)
    keep = gy.clone()
    r = torch.zeros(shape, dtype=BF, device=DEV, requires_grad=True)
    q = torch.zeros((4, 48), dtype=BF, device=DEV, requires_grad=True)
    ref_r, ref_q = torch.zeros_like(gy), torch.zeros_like(gy)      # the same additions in the same order
    for _ in range(4):
        y = nv.nvfp4_linear_train(x, w, residual=r, **kw)
        (y + q).backward(gy)
        y = nv.nvfp4_linear_train(x, w, residual=r, **kw)
        y.backward(gy)
        ref_q += keep
        ref_r += keep
        ref_r += keep
        assert torch.equal(gy, keep) and torch.equal(q.grad, ref_q)
        assert r.grad.shape == r.shape and torch.equal(r.grad.view(4, 48), ref_r)
    assert len({t.data_ptr() for t in (r.grad, q.grad, gy)}) == 3
