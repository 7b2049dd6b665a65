"""Layer norm with the residual's addition: every output form bit for bit against the oracle
(statistics in float64, prescribed roundings), the gradient against the float64 formula and
against differences, refusals, streams and graph replays; and the RMS norm's 8-bit codes."""
import numpy as np
import pytest
import torch

import oracle as o
import workloads
from tests._util import layout_to_canonical, oracle_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
TYPES = [(BF, None, BF), (BF, BF, BF), (BF, F, F), (F, None, BF), (F, F, F), (BF, BF, F)]
SHAPES = [(1, 16), (5, 16), (3, 48), (67, 128), (2, 144), (33, 1024), (9, 1040), (4, 2064), (7, 5120), (2, 8192),
          (3, 16384)]


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


def _f(t):
    return t.detach().float().cpu().numpy()


def _dev(*ts):
    return tuple(None if t is None else t.to(DEV) for t in ts)


def _inputs(m, k, xd, rd, wd, seed=0, bias=True):
    """x, residual (None for rd None), weight and bias: outliers, means away from zero, and where
    there are rows enough one of zeros, one of a constant, tiny and huge ones, and one whose first
    value (the pivot) is the outlier."""
    x = workloads.draw("normal_outliers", (m, k), 160 + seed, 0).float()
    x += workloads.draw("normal", (m, 1), 164 + seed, 4).float()
    if m > 2:
        x[1] = 0.0
        x[2] *= 1e-20
    if m > 3:
        x[3] *= 1e15
    if m > 4:
        x[4] = 7.0
    if m > 5:
        x[5, 0] = 3e4
    if m > 6:
        x[6] = x[6] * 1e-2 + 100.0
    res = None
    if rd is not None:
        res = workloads.draw("t3", (m, k), 161 + seed, 1).float() * 1.37
        if m > 2:
            res[1] = 0.0
            res[2] *= 1e-20
        if m > 4:
            res[4] = -2.5
        if rd == F:
            res = res * (1 + 2.0 ** -13)
        res = res.to(rd)
    if xd == F:
        x = x * (1 + 2.0 ** -12)
    w = 1.0 + 0.1 * workloads.draw("normal", (k,), 162 + seed, 2).float()
    b = 0.1 * workloads.draw("normal", (k,), 163 + seed, 3).float()
    return x.to(xd), res, w.to(wd), b.to(wd) if bias else None


def _oracle(x, res, w, b, eps):
    return o.layernorm(_f(x), _f(w), None if b is None else _f(b), eps, None if res is None else _f(res),
                       "f32" if res is not None and res.dtype == F else "bf16")


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("xd,rd,wd", TYPES)
def test_outputs_bitwise(m, k, xd, rd, wd):
    x, res, w, b = _inputs(m, k, xd, rd, wd, m + k, bias=(m + k) % 3 != 0)
    r_ref, y_ref = _oracle(x, res, w, b, 1e-6)
    xg, rg, wg, bg = _dev(x, res, w, b)
    got = nv().layernorm(xg, wg, bg, 1e-6, rg)
    y = got if res is None else got[0]
    assert y.dtype == BF and np.array_equal(_f(y), y_ref)
    if res is not None:
        assert got[1].dtype == rd and np.array_equal(_f(got[1]), r_ref)
    got = nv().layernorm_checkpoint(xg, wg, bg, 1e-6, rg)
    assert torch.equal(got[0], y)
    codes, scales = o.checkpoint_pack(y_ref)
    assert np.array_equal(got[-1].codes.cpu().numpy(), codes) and np.array_equal(got[-1].scales.cpu().numpy(), scales)
    # 8-bit block codes: those of y
    got = nv().fp8_quantize_layernorm(xg, wg, bg, 1e-6, rg)
    codes, scales = o.fp8_quantize(y_ref, 1)
    assert np.array_equal(got[0].cpu().numpy(), codes) and np.array_equal(got[1].cpu().numpy(), scales.T)
    if res is not None:
        assert np.array_equal(_f(got[2]), r_ref)
    # NVFP4 codes under the dynamic scale and a static one
    for static in (None, 3.0):
        got = nv().quantize_layernorm(xg, wg, bg, 1e-6, rg, static)
        gsf = np.float32(o.global_sf(o.amax(y_ref))) if static is None else np.float32(static)
        assert float(got[2]) == float(gsf)
        packed, sc = oracle_quantize(y_ref, gsf)
        assert np.array_equal(got[0].cpu().numpy(), packed)
        assert np.array_equal(layout_to_canonical(got[1].cpu().numpy(), m, k), sc)
        if res is not None:
            assert np.array_equal(_f(got[3]), r_ref)


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("xd,rd,wd", TYPES)
def test_rmsnorm_fp8_is_its_own_output_quantized(m, k, xd, rd, wd):
    x, res, w, _ = _inputs(m, k, xd, rd, wd, m + k)
    xg, rg, wg = _dev(x, res, w)
    plain = nv().rmsnorm(xg, wg, 1e-6, rg)
    got = nv().fp8_quantize_rmsnorm(xg, wg, 1e-6, rg)
    codes, scales = nv().fp8_quantize_activation(plain if res is None else plain[0])
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
    if res is not None:
        assert torch.equal(got[2], plain[1])


def test_rows_past_the_grid_and_long_offsets():
    # 2^31 values and more, in every one-pass form: the last rows against the oracle
    m, k = 2 ** 31 // 16384 + 3, 16384
    x = torch.randn(64, k, generator=torch.Generator().manual_seed(1)).to(BF)
    xg = x.to(DEV).repeat(m // 64 + 1, 1)[:m]
    w = torch.ones(k, device=DEV)
    y = nv().layernorm(xg, w)
    rows = [0, 63, m - 2, m - 1]
    _, ref = o.layernorm(_f(xg[rows]), np.ones(k), None, 1e-6)
    assert np.array_equal(_f(y[rows]), ref)
    del y
    codes, scales = nv().fp8_quantize_layernorm(xg, w)
    c, s = o.fp8_quantize(ref, 1)
    assert np.array_equal(codes[rows].cpu().numpy(), c) and np.array_equal(scales[:, rows].cpu().numpy(), s.T)


def test_special_values():
    x = torch.randn(6, 64, generator=torch.Generator().manual_seed(2))
    x[1, 5] = float("inf")
    x[2, 0] = float("nan")
    x[3] = 0.0
    x[4] = 2.0
    w, b = torch.ones(64), torch.full((64,), 0.5)
    xg, wg, bg = _dev(x, w, b)
    y = nv().layernorm(xg, wg, bg)
    assert y[1].isnan().all() and y[2].isnan().all()
    assert (y[3:5] == 0.5).all() and y[[0, 5]].isfinite().all()
    codes, _ = nv().fp8_quantize_layernorm(xg, wg, bg)
    assert ((codes[1:3] & 0x7F) == 0x7F).all() and ((codes[[0, 3, 4, 5]] & 0x7F) != 0x7F).all()
    # a constant row without an eps: 0 times infinity, as the formula says
    assert nv().layernorm(xg[4:5], wg, bg, 0.0).isnan().all()


def _grad_reference(gy, r, w, eps, gres):
    return o.layernorm_grads(_f(gy), _f(r), _f(w), eps, None if gres is None else _f(gres))


def _check_grads(got, gy, r, w, eps, gres, m, k):
    """fp32 steps: a value of grad_r is s (g - f1 - n f2) + grad_residual: each of the terms rounds
    a handful of times to 2^-24 of itself, and f1 and f2 come from lanes' fp32 sums of 16 products
    (whose magnitudes the means of |g| and |g d| bound, d the distance from the pivot, at most
    |n| + |n_0| in units of the spread).  grad_w and grad_b are sums over rows in fp32."""
    gr, gw, gb = _grad_reference(gy, r, w, eps, gres)
    g64, r64, w64 = (_f(t).astype(np.float64) for t in (gy, r, w))
    c = r64 - r64.mean(-1, keepdims=True)
    s = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    n, g = c * s, g64 * w64
    mg = np.abs(g).mean(-1, keepdims=True)
    mgd = (np.abs(g) * (np.abs(n) + np.abs(n[:, :1]))).mean(-1, keepdims=True) + np.abs(n[:, :1]) * mg
    bound = U * s * (8 * np.abs(g) + 24 * mg + np.abs(n) * 32 * mgd)
    if gres is not None:
        bound = bound + U * np.abs(_f(gres))
    bound = bound + np.abs(gr) * (2.0 ** -8 if r.dtype == BF else U) + 1e-37
    assert np.all(np.abs(_f(got[0]) - gr) <= bound)
    rows = U * (m + 8)
    assert np.all(np.abs(_f(got[1]) - gw) <= rows * (np.abs(g64 * n)).sum(0) + 1e-37)
    assert np.all(np.abs(_f(got[2]) - gb) <= rows * np.abs(g64).sum(0) + 1e-37)


@pytest.mark.parametrize("m,k", SHAPES + [(700, 256), (1500, 1040)])
@pytest.mark.parametrize("rd,wd,res", [(BF, BF, False), (BF, F, True), (F, F, True), (F, BF, False)])
def test_gradient(m, k, rd, wd, res):
    r, _, w, _ = _inputs(m, k, rd, None, wd, m)
    if m > 3:
        r[3] *= 1e-15     # magnitudes whose gradient fp32 holds: the extremes have their own test
    gy = workloads.draw("t3", (m, k), 170, m, 1e-2)
    gres = workloads.draw("normal", (m, k), 171, m, 1e-2).to(rd) if res else None
    got = nv().layernorm_backward(*_dev(gy, r, w), 1e-6, *_dev(gres))
    assert got[0].dtype == rd and got[1].dtype == got[2].dtype == F
    _check_grads(got, gy, r, w, 1e-6, gres, m, k)
    again = nv().layernorm_backward(*_dev(gy, r, w), 1e-6, *_dev(gres))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradient_against_differences():
    m, k, h = 3, 48, 1e-2
    g = torch.Generator().manual_seed(7)
    r, w = torch.randn(m, k, generator=g), 1 + 0.1 * torch.randn(k, generator=g)
    gy = torch.randn(m, k, generator=g).to(BF)
    gr, gw, gb = (t.cpu().double() for t in nv().layernorm_backward(*_dev(gy, r, w), 1e-3))

    def f(r, w, b):
        return (gy.double() * torch.nn.functional.layer_norm(r.double(), (k,), w.double(), b.double(), 1e-3)).sum()

    b = torch.zeros(k)
    for i in (0, 13, 47):
        e, d = torch.zeros(m, k), torch.zeros(k)
        e[1, i] = d[i] = h
        # central differences: h^2 / 6 times third derivatives of a few units
        assert abs((f(r.double() + e, w, b) - f(r.double() - e, w, b)) / (2 * h) - gr[1, i]) < 2e-3
        assert abs((f(r, w + d.double(), b) - f(r, w - d.double(), b)) / (2 * h) - gw[i]) < 1e-4
        assert abs((f(r, w, b + d.double()) - f(r, w, b - d.double())) / (2 * h) - gb[i]) < 1e-4


def test_gradient_extremes():
    # rows from 1e-15 to 1e15, an odd count over several workgroups; eps 0 with rows beyond the last
    m, k = 37, 1040
    r = torch.randn(m, k, generator=torch.Generator().manual_seed(3)) * torch.logspace(-15, 15, m)[:, None]
    gy, w = workloads.draw("normal", (m, k), 172, 0), torch.ones(k)
    got = nv().layernorm_backward(*_dev(gy, r, w), 0.0)
    _check_grads(got, gy, r, w, 0.0, None, m, k)
    # no rows at all
    got = nv().layernorm_backward(torch.empty(0, 64, device=DEV, dtype=BF), torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV))
    assert got[0].shape == (0, 64) and not got[1].any() and not got[2].any()


def test_empty_strided_and_misaligned():
    w, b = torch.ones(64, device=DEV), torch.zeros(64, device=DEV)
    assert nv().layernorm(torch.empty(0, 64, device=DEV, dtype=BF), w, b).shape == (0, 64)
    codes, scales = nv().fp8_quantize_layernorm(torch.empty(0, 64, device=DEV, dtype=BF), w, b)
    assert codes.shape == (0, 64) and scales.shape == (1, 0)
    x = torch.randn(5, 2, 3, 128, device=DEV).to(BF)
    want = nv().layernorm(x[..., :64].contiguous(), w, b)
    assert torch.equal(nv().layernorm(x[..., :64], w, b), want) and want.shape == (5, 2, 3, 64)
    flat = torch.empty(30 * 64 + 1, device=DEV, dtype=BF)
    flat[1:] = x[..., :64].reshape(-1)
    assert torch.equal(nv().layernorm(flat[1:].view(5, 2, 3, 64), w, b), want)
    assert torch.equal(nv().layernorm(x[..., :64].transpose(0, 1), w, b), want.transpose(0, 1))


def test_refusals():
    x, w, b = (torch.ones(s, device=DEV, dtype=BF) for s in ((4, 64), (64,), (64,)))
    for bad in (lambda: nv().layernorm(x[:, :24].contiguous(), w[:24].contiguous()), lambda: nv().layernorm(x, w[:48]),
                lambda: nv().layernorm(x, w, b[:48]), lambda: nv().layernorm(x, w, b.float()),
                lambda: nv().layernorm(x.half(), w), lambda: nv().layernorm(x, w, b, -1.0),
                lambda: nv().layernorm(x, w, b.cpu()), lambda: nv().layernorm(x, w, b, 1e-6, x[:2]),
                lambda: nv().layernorm(x.float(), w, b, 1e-6, x),
                lambda: nv().layernorm(torch.ones(1, 16400, device=DEV), torch.ones(16400, device=DEV)),
                lambda: nv().layernorm_backward(x, x[:2], w), lambda: nv().layernorm_backward(x, x, w, 1e-6, x.float()),
                lambda: nv().layernorm_backward(x.float(), x, w)):
        with pytest.raises(ValueError):
            bad()


def test_training_form():
    m, k = 45, 1040
    x, res, w, b = _inputs(m, k, BF, F, F, 5)
    x[2:4], res[2:4] = x[0:2], res[0:2]     # magnitudes of one
    xg, rg, wg, bg = _dev(x, res, w, b)
    leaves = [t.clone().requires_grad_() for t in (xg, rg, wg, bg)]
    y, r, ck = nv().layernorm_train(leaves[0], leaves[2], leaves[3], 1e-6, leaves[1], checkpoint=True)
    want = nv().layernorm_checkpoint(xg, wg, bg, 1e-6, rg)
    assert torch.equal(y, want[0]) and torch.equal(r, want[1]) and torch.equal(ck.codes, want[2].codes)
    gy, gr = torch.randn_like(y), torch.randn_like(r)
    torch.autograd.backward((y, r), (gy, gr))
    gx, gw, gb = nv().layernorm_backward(gy, want[1], wg, 1e-6, gr)
    assert torch.equal(leaves[0].grad, gx.to(BF)) and torch.equal(leaves[1].grad, gx)
    assert torch.equal(leaves[2].grad, gw) and torch.equal(leaves[3].grad, gb)
    # only the stream, only y, no bias
    x1 = xg.clone().requires_grad_()
    nv().layernorm_train(x1, wg, None, 1e-6, rg)[1].sum().backward()
    assert (x1.grad == 1).all()
    x1 = xg.clone().requires_grad_()
    nv().layernorm_train(x1, wg)[0].sum().backward()
    assert x1.grad.shape == x1.shape
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(nv().layernorm_train(x1, wg).float().square().sum(), x1, create_graph=True)
        g.sum().backward()


def test_streams_and_graph():
    m, k = 33, 1024
    x, res, w, b = _dev(*_inputs(m, k, BF, BF, F, 9))
    gy = torch.randn(m, k, device=DEV).to(BF)

    def all_forms():
        return (*nv().layernorm_checkpoint(x, w, b, 1e-6, res)[:2], *nv().quantize_layernorm(x, w, b, 1e-6, res),
                *nv().fp8_quantize_layernorm(x, w, b, 1e-6, res), *nv().layernorm_backward(gy, x, w, 1e-6, res))

    want = [t.clone() for t in all_forms()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_forms()
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_forms()
    for i in range(3):
        x.copy_(torch.randn(m, k, device=DEV))
        want = [t.clone() for t in all_forms()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), i


@pytest.mark.parametrize("m,k", [(5, 64), (9, 1040), (600, 1040), (7, 5120), (1100, 5120), (2, 16384)])
def test_residual_sum_in_place(m, k):
    # the C calls may write r over the residual, or over x of its type: the pivot is read before
    import nvfp4_w4a4_quantized_global_amd._lib as L
    x, res, w, b = _dev(*_inputs(m, k, BF, BF, F))
    y, r = nv().layernorm(x, w, b, 1e-6, res)
    codes, scales, _ = nv().fp8_quantize_layernorm(x, w, b, 1e-6, res)
    s = torch.cuda.current_stream().cuda_stream
    for over in (0, 1):
        a = [x.clone(), res.clone()]
        got = torch.empty_like(y)
        L.check(L.lib().nvfp4_layernorm(a[0].data_ptr(), 0, a[1].data_ptr(), 0, w.data_ptr(), b.data_ptr(), 1, m, k, 1e-6,
                                        a[over].data_ptr(), got.data_ptr(), None, None, s))
        assert torch.equal(got, y) and torch.equal(a[over], r) and torch.equal(a[1 - over], (x, res)[1 - over])
        a = [x.clone(), res.clone()]
        c, sc = torch.empty_like(codes), torch.empty_like(scales)
        L.check(L.lib().nvfp4_fp8_quantize_layernorm(a[0].data_ptr(), 0, a[1].data_ptr(), 0, w.data_ptr(), b.data_ptr(), 1, m,
                                                     k, 1e-6, a[over].data_ptr(), c.data_ptr(), sc.data_ptr(), s))
        assert torch.equal(c, codes) and torch.equal(sc, scales) and torch.equal(a[over], r)
