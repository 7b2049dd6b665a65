"""Calls of the layer norm and the 8-bit blocks that their documentation allows and that are easily
missed: more rows than a launch has workgroups, rows that are not finite in front of 4-bit codes,
calls on two streams at once."""
import pytest
import torch

import workloads
from tests.test_gpu_fp8 import nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _rows(m, k, seed, period=1009):
    g = torch.Generator(device=DEV).manual_seed(seed)
    block = torch.randn((period, k), generator=g, device=DEV).to(BF)
    return block.repeat(-(-m // period), 1)[:m]


def _bits(t):
    return t if t.dtype == torch.uint8 else t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


# rows of 16 values go 32 to a workgroup, of 1040 one to each: both past 2^20 workgroups
@pytest.mark.parametrize("m,k", [(32 * 2 ** 20 + 77, 16), (2 ** 20 + 77, 1040)])
def test_more_rows_than_workgroups(m, k):
    x = _rows(m, k, 1)
    w, b = (1 + 0.1 * torch.randn(k, device=DEV)), 0.1 * torch.randn(k, device=DEV)
    pick = torch.tensor([*range(40), *range(m - 120, m)], device=DEV)
    some = x[pick]
    got, want = nv().layernorm_checkpoint(x, w, b), nv().layernorm_checkpoint(some, w, b)
    assert torch.equal(got[0][pick], want[0]) and torch.equal(got[1].codes[pick], want[1].codes)
    assert torch.equal(got[1].scales[pick], want[1].scales)
    del got
    for form, args in ((nv().fp8_quantize_layernorm, (w, b)), (nv().fp8_quantize_rmsnorm, (w,)),
                       (nv().fp8_quantize_activation, ())):
        (codes, scales), (c, s) = form(x, *args), form(some, *args)
        assert torch.equal(codes[pick], c) and torch.equal(scales[:, pick], s)
    codes, scales, _ = nv().quantize_layernorm(x, w, b, global_sf_x=30.0)
    c, s, _ = nv().quantize_layernorm(some, w, b, global_sf_x=30.0)
    kt = -(-k // 128)
    assert torch.equal(codes[pick], c) and torch.equal(scales.view(kt, m, 8)[:, pick], s.view(kt, len(pick), 8))
    r, gy = x, _rows(m, k, 2, 1013)
    gr, gw, gb = nv().layernorm_backward(gy, r, w)
    assert torch.equal(gr[pick], nv().layernorm_backward(gy[pick], some, w)[0])
    assert gw.isfinite().all() and gb.isfinite().all()


def test_more_values_than_threads_times_sixteen():
    m, k = 262400, 16384
    codes = torch.randint(0, 127, (1009, k), device=DEV, dtype=torch.uint8).repeat(-(-m // 1009), 1)[:m].contiguous()
    scales = torch.rand(k // 128, m, device=DEV) + 0.5
    v = nv().fp8_dequantize(codes, scales)
    for p in (slice(0, 64), slice(2 ** 32 // k - 32, 2 ** 32 // k + 32), slice(m - 64, m)):
        assert torch.equal(v[p], nv().fp8_dequantize(codes[p], scales[:, p].contiguous()))


@pytest.mark.parametrize("m,k", [(1, 144), (1, 5120), (6, 64), (40, 1040), (7, 5120), (5, 16384)])
@pytest.mark.parametrize("static", [None, 25.0])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_that_are_not_finite_in_front_of_4_bit_codes(m, k, static, residual):
    """The codes of quantize_activation on the norm's output under the same scale, whatever is in the rows."""
    x = workloads.draw("normal_outliers", (m, k), 360, m).float()
    x[0, k // 2] = float("inf")
    if m > 3:
        x[1, 0], x[2, -1], x[3, 3] = float("nan"), float("-inf"), float("nan")
    x = x.to(BF).to(DEV)
    w, b = (1 + 0.1 * torch.randn(k, device=DEV)), 0.1 * torch.randn(k, device=DEV)
    res = workloads.draw("t3", (m, k), 361, m).to(DEV) if residual else None
    y = nv().layernorm(x, w, b, 1e-6, res)
    y = y if res is None else y[0]
    assert y[0].isnan().all()
    got = nv().quantize_layernorm(x, w, b, 1e-6, res, static)
    if static is None and m > 4:
        # an input with NaN has no defined dynamic scale for the quantizer: the norm's rows that are
        # finite give it here
        fine = y[y.isfinite().all(-1)]
        assert torch.equal(got[2], nv().quantize_activation(fine)[2])
    want = nv().quantize_activation(y, got[2])
    for a, c in zip(got[:3], want):
        assert torch.equal(_bits(a.reshape(-1)), _bits(c.reshape(-1)))
    codes, scales = nv().fp8_quantize_layernorm(x, w, b, 1e-6, res)[:2]
    c, s = nv().fp8_quantize_activation(y)
    assert torch.equal(codes, c) and torch.equal(scales, s)


def test_two_streams_at_once():
    """Products whose tiles are split along K, norms with a second pass and gradients, interleaved on two
    streams: each call has a workspace of its own."""
    shapes = [(130, 5120, 256), (64, 25600, 512), (1, 5120, 1024), (16, 2064, 333)]
    work = []
    for i, (m, k, n) in enumerate(shapes * 2):
        x = workloads.draw("normal", (m, k), 370 + i, m).to(DEV)
        wq = nv().fp8_quantize_weight(workloads.draw("normal", (n, k), 380 + i, n, 0.05).to(DEV))
        ln = torch.ones(min(k, 16384), device=DEV)
        h = x[:, :min(k, 16384)].contiguous()

        def calls(x=x, wq=wq, ln=ln, h=h):
            return [nv().fp8_linear(x, *wq), *nv().quantize_layernorm(h, ln), *nv().layernorm_backward(h, h, ln),
                    nv().fp8_quantize_activation(x, column_sum=True)[2]]
        work.append(calls)
    want = [[t.clone() for t in c()] for c in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(4):
        for i, c in enumerate(work):
            with torch.cuda.stream(streams[(i + turn) % 2]):
                got.append((i, c()))
    torch.cuda.synchronize()
    for i, ts in got:
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(ts, want[i]))
