"""The layer norm's gradient over the whole range of its rows: magnitudes whose products with the
gradient leave fp32's range while the gradient itself is an fp32 number, also where the row's first
value is by far its largest.  Against the float64 formula, with the bounds of its fp32 steps."""
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


def _check(got, gy, r, w, eps, gres):
    """Row sums are taken in fp64, of the products g = gy w rounded to fp32; every other step of
    s (g - f1 - n f2) + grad_residual rounds to 2^-24 of its result: s, the centred value, n (after three
    roundings), f1 = mean g, f2 = mean g n, g - f1, n f2, their difference, its product with s and the
    last addition: at most six of them on the way of |g|, eight of mean |g|, twelve of |n| mean |g n|.
    fp64 sums of at most 32 steps in a row, and their cancellation against the pivot p, leave the centred
    value and the sum of g (r - mu) off by 2^-53 32 (mean |r - p| + |mu|) and the same with |g|.  A step whose
    result is subnormal is off by 2^-150 absolutely.  grad_w and grad_b are sums over rows."""
    m = r.shape[0]
    ref = o.layernorm_grads(_f(gy), _f(r), _f(w), eps, None if gres is None else _f(gres))
    gy64, r64, w64 = (_f(t).astype(np.float64) for t in (gy, r, w))
    mean = lambda a: np.mean(a, -1, keepdims=True)  # noqa: E731
    mu = mean(r64)
    c = r64 - mu
    s = 1.0 / np.sqrt(mean(c * c) + np.float64(np.float32(eps)))
    n, g = np.abs(c) * s, np.abs(gy64 * w64)
    mg, mgn = mean(g), mean(g * n)
    apart = np.abs(r64 - r64[:, :1])
    e64 = 2.0 ** -48
    n_off = e64 * s * (mean(apart) + np.abs(mu))
    f2_off = e64 * s * (mean(g * apart) + mean(apart) * mg)
    tol = s * (U * (6 * g + 8 * mg + 12 * n * mgn) + n_off * mgn + n * f2_off) + 2.0 ** -150 * (4 + n + s * (1 + n) * (1 + mg))
    if gres is not None:
        tol = tol + U * np.abs(_f(gres)).astype(np.float64)
    if r.dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(ref[0]) + tol) + 2.0 ** -134
    bad = ~(np.abs(_f(got[0]).astype(np.float64) - ref[0]) <= tol)
    assert not bad.any(), f"rows {np.flatnonzero(bad.any(-1))}: {_f(got[0])[bad][:4]} for {ref[0][bad][:4]}"
    terms = np.abs(gy64) * (n + n_off)
    assert np.all(np.abs(_f(got[1]).astype(np.float64) - ref[1]) <= U * (m + 4) * terms.sum(0) + (np.abs(gy64) * n_off).sum(0) + 2.0 ** -150 * m)
    assert np.all(np.abs(_f(got[2]).astype(np.float64) - ref[2]) <= U * (m + 4) * np.abs(gy64).sum(0) + 2.0 ** -150 * m)


# rms of the rows; values to five times that, whose reciprocals are normal fp32 numbers
RMS = [1.0, 1e-10, 1e-15, 1e10, 1e15, 1e19, 1e22, 1e23, 1e27, 1e31, 1e34, 1e36, 1e37]


@pytest.mark.parametrize("k", [48, 1024, 1040, 5120])
@pytest.mark.parametrize("rd,wd", [(BF, F), (F, F), (F, BF)])
@pytest.mark.parametrize("eps,correlated,gres,scale", [(1e-6, True, False, 20.0), (1e-6, False, True, 1.0), (0.0, True, False, 1.0)])
def test_gradient_of_rows_of_any_size(k, rd, wd, eps, correlated, gres, scale):
    """Gradients that follow r (most of s g is then projected away) and gradients that do not; with
    eps = 0 rows down to 1e-30 as well."""
    rms = np.array(RMS + ([1e-20, 1e-23, 1e-30] if eps == 0.0 else [1e-20, 1e-30]))
    m = len(rms)
    base = workloads.draw("normal", (m, k), 300 + k, 0).double()
    r = (base * torch.from_numpy(rms)[:, None]).to(rd)
    w = (1.0 + 0.1 * workloads.draw("normal", (k,), 301, 1).float()).to(wd)
    gy = workloads.draw("normal", (m, k), 302, 2).double()
    if correlated:
        gy = base + 0.1 * gy
    gy = (gy * scale).to(BF)
    extra = workloads.draw("normal", (m, k), 303, 3, 1e-2).to(rd) if gres else None
    got = nv().layernorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), eps, None if extra is None else extra.to(DEV))
    _check(got, gy, r, w, eps, extra)


@pytest.mark.parametrize("m,k", [(6, 48), (9, 1040), (7, 5120), (6, 16384)])
@pytest.mark.parametrize("rd", [BF, F])
@pytest.mark.parametrize("large", [3e4, 1e20, 3e36, -8e37])
def test_a_first_value_far_from_the_others(m, k, rd, large):
    """The sums are taken around the row's first value: here the largest of all, or far from the mean,
    beside gradients of 20, of 1e-3 and of 1e30."""
    r = workloads.draw("normal", (m, k), 310 + m, 0).float()
    r[0, 0], r[1, 0], r[2, 0], r[2, -1], r[3, 0] = large, large, large, large, large
    r[3, 1:] *= abs(large) * 1e-6
    r = r.to(rd)
    w = 1.0 + 0.1 * workloads.draw("normal", (k,), 311, 1).float()
    gy = workloads.draw("normal", (m, k), 312, 2).float()
    gy[0] = 20.0
    gy[1] *= 1e-3
    gy[2] *= 20.0
    if abs(large) > 1e6:
        gy[3] *= 1e30
    gy = gy.to(BF)
    _check(nv().layernorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), 1e-6), gy, r, w, 1e-6, None)


def test_repeats_bit_for_bit_at_the_extremes():
    m, k = 40, 1040
    r = workloads.draw("normal", (m, k), 320, 0).float() * torch.logspace(-30, 36, m)[:, None]
    gy, w = workloads.draw("normal", (m, k), 321, 1).to(DEV), torch.ones(k, device=DEV)
    a, b = (nv().layernorm_backward(gy, r.to(DEV), w, 0.0) for _ in range(2))
    assert all(torch.equal(x, y) and x.isfinite().all() for x, y in zip(a, b))


@pytest.mark.parametrize("k", [48, 1040, 16384])
@pytest.mark.parametrize("at", [0, -1])
def test_the_largest_gradients(k, at):
    """|grad_y w| up to 1e36, with the signs of the row and half its spread in one value: n mean(g n) is then
    as large as it gets, sqrt(k) / 2 times the gradient."""
    m = 3
    r = torch.sign(workloads.draw("normal", (m, k), 330, k).float() + 1e-3)
    r[:, at] = k ** 0.5
    r *= torch.tensor([1e3, 1e10, 1e30])[:, None]
    gy = (9.8e35 * torch.sign(r - r.mean(-1, keepdim=True))).to(BF)
    w = torch.ones(k)
    assert float(gy.float().abs().max()) < 1e36
    got = nv().layernorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), 1e-6)
    assert got[0].isfinite().all()
    _check(got, gy, r, w, 1e-6, None)
