"""The RMS norm's gradient over the whole range of its stream: rows whose squares, or whose
products with the gradient, leave fp32's range while the gradient itself is an fp32 number.
Against the float64 formula, with the bounds of its fp32 steps."""
import numpy as np
import pytest
import torch

import oracle as o
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


def _f(t):
    return t.detach().float().cpu().numpy()


def _bounds(gy, r, w, eps, gres, rows):
    """Every fp32 step rounds to 2^-24 of its result: s, g = gy w, n = r s, the projection factor f and
    the products with them, at most eight on the way of s g or of n f.  d = sum(g r) carries the rounding of
    each g (and, were it summed in fp32, 40 more): 50 in all of sum |g r|.  A step whose result is
    subnormal is off by 2^-150 absolutely: of f times |n|, of the others as they are.  grad_w: a
    term gy n carries three roundings, its sum over the rows one an addition."""
    gy, r, w = (np.asarray(a, dtype=np.float64) for a in (gy, r, w))
    k = r.shape[1]
    s = 1.0 / np.sqrt(np.mean(r * r, -1, keepdims=True) + np.float64(np.float32(eps)))
    n = np.abs(r) * s
    g = np.abs(gy * w)
    d = np.sum(np.abs(gy * w * r), -1, keepdims=True)
    q = 0.0 if gres is None else np.abs(np.asarray(gres, dtype=np.float64))
    tol_r = U * (8 * (s * g + q) + 50 * n * s * (s * (d / k))) + 2.0 ** -150 * (4 + n)
    tol_w = U * (rows + 4) * np.sum(np.abs(gy) * n, 0) + 2.0 ** -150 * rows
    return tol_r, tol_w


# rms of the rows; each fits the stream, its reciprocal is a normal fp32 number
RMS = [1.0, 1e-10, 1e-15, 1e10, 1e15, 1e19, 1e22, 1e23, 1e27, 1e31, 1e34, 1e36]


@pytest.mark.parametrize("k", [48, 1024, 1040, 5120])
@pytest.mark.parametrize("rd,wd", [(BF, F), (F, F), (F, BF)])
@pytest.mark.parametrize("eps,correlated,gres", [(1e-6, True, False), (1e-6, False, True), (0.0, True, False)])
def test_gradient_of_rows_of_any_size(k, rd, wd, eps, correlated, gres):
    """Gradients that follow r (sum(g r) is then as large as it gets and most of s g is projected
    away) and gradients that do not; with eps = 0 rows down to 1e-30 as well."""
    rms = np.array(RMS + ([1e-20, 1e-23, 1e-30] if eps == 0.0 else [1e-20, 1e-30]))
    m = len(rms)
    base = workloads.draw("normal", (m, k), 200 + k, 0).double()
    r = (base * torch.from_numpy(rms)[:, None]).to(rd)
    w = (1.0 + 0.1 * workloads.draw("normal", (k,), 201, 1).float()).to(wd)
    gy = workloads.draw("normal", (m, k), 202, 2).double()
    if correlated:
        gy = base + 0.1 * gy
    gy = gy.to(BF)
    extra = workloads.draw("normal", (m, k), 203, 3, 1e-2).to(rd) if gres else None
    gx, gw = nv().rmsnorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), eps, None if extra is None else extra.to(DEV))
    e = None if extra is None else _f(extra)
    ref_x, ref_w = o.rmsnorm_grads(_f(gy), _f(r), _f(w), eps, e)
    tol_r, tol_w = _bounds(_f(gy), _f(r), _f(w), eps, e, m)
    if rd == BF:
        tol_r = tol_r + 2.0 ** -8 * (np.abs(ref_x) + tol_r) + 2.0 ** -134
    bad = ~(np.abs(_f(gx) - ref_x) <= tol_r)
    assert not bad.any(), f"rows of rms {rms[bad.any(-1)]}"
    assert np.all(np.abs(_f(gw) - ref_w) <= tol_w)


@pytest.mark.parametrize("m,k", [(6, 48), (9, 1040), (7, 5120), (3, 16384)])
@pytest.mark.parametrize("rd", [BF, F])
def test_zero_tiny_and_large_rows_among_ordinary_ones(m, k, rd):
    """A zero row, one of 1e-20 and one of 1e15 beside rows with outliers, under a usual eps."""
    r = workloads.draw("normal_outliers", (m, k), 210 + m, 0).float()
    r[0], r[1], r[2] = 0.0, r[1] * 1e-20, r[2] * 1e15
    r = r.to(rd)
    w = 1.0 + 0.1 * workloads.draw("normal", (k,), 211, 1).float()
    gy = workloads.draw("normal", (m, k), 212, 2, 1e-2)
    gx, gw = nv().rmsnorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), 1e-6)
    ref_x, ref_w = o.rmsnorm_grads(_f(gy), _f(r), _f(w), 1e-6)
    tol_r, tol_w = _bounds(_f(gy), _f(r), _f(w), 1e-6, None, m)
    if rd == BF:
        tol_r = tol_r + 2.0 ** -8 * (np.abs(ref_x) + tol_r) + 2.0 ** -134
    assert np.all(np.abs(_f(gx) - ref_x) <= tol_r)
    assert np.all(np.abs(_f(gw) - ref_w) <= tol_w)
