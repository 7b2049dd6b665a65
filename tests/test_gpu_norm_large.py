"""The norm's weight gradient over more than 2^31 values: a row that is skipped, read twice or
taken from elsewhere changes the sum."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
U = 2.0 ** -24


@pytest.mark.parametrize("rd", [BF, torch.float32])
def test_weight_gradient_past_2_31_values(rd):
    import nvfp4_w4a4_quantized_global_amd as nv
    m, k = 131500, 16384
    last = m - 2 ** 31 // k                       # rows past the 2^31st value
    assert last > 400
    g = torch.Generator(device=DEV).manual_seed(3)
    r, gy = torch.empty((m, k), dtype=rd, device=DEV), torch.empty((m, k), dtype=BF, device=DEV)
    block = torch.randn((1500, k), generator=g, device=DEV)
    for i in range(0, m, 1500):                   # every block of rows differs from the others
        n = min(1500, m - i)
        r[i:i + n] = block[:n] * (1.0 + (i // 1500) * 0.125)
        gy[i:i + n] = block[:n] * (0.5 + (i // 1500) % 5)
    gy[-last:] *= 16.0
    w = torch.ones(k, device=DEV)
    _, gw = nv.rmsnorm_backward(gy, r, w, 1e-6)
    ref, mag = (torch.zeros(k, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, m, 1500):
        rb, gb = r[i:i + 1500].double(), gy[i:i + 1500].double()
        t = gb * rb / torch.sqrt(rb.square().mean(1, keepdim=True) + float(torch.tensor(1e-6)))
        ref += t.sum(0)
        mag += t.abs().sum(0)
    # three roundings of a term; additions on its way: its workgroup's rows (512 workgroups walk them), then
    # the workgroups' partials in 32 interleaved sets of 16, then the sets
    tol = U * (3 + -(-m // 512) + 16 + 32) * mag
    assert bool(((gw.double() - ref).abs() <= tol).all())
