"""RMS norm with the residual's addition: every output form bit for bit against the oracle
(fp64 mean square, prescribed roundings), the gradient against the float64 formula and
against differences, refusals, streams and graph replays."""
import numpy as np
import pytest
import torch

import oracle as o
import workloads
from tests._util import layout_to_canonical, oracle_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


def _f(t):
    return t.detach().float().cpu().numpy()


def _inputs(m, k, xd, rd, wd, seed=0):
    """x, residual (None for rd None) and weight; outlier activations, a zero row when there
    are several, tiny and huge values."""
    x = workloads.draw("normal_outliers", (m, k), 60 + seed, 0).float()
    if m > 2:
        x[1] = 0.0
        x[2] *= 1e-20
    if m > 3:
        x[3] *= 1e15
    res = None
    if rd is not None:
        res = workloads.draw("t3", (m, k), 61 + seed, 1).float() * 1.37
        if m > 2:
            res[1] = 0.0
            res[2] *= 1e-20
        if rd == torch.float32:
            res = res * (1 + 2.0 ** -13)
        res = res.to(rd)
    if xd == torch.float32:
        x = x * (1 + 2.0 ** -12)
    w = 1.0 + 0.1 * workloads.draw("normal", (k,), 62 + seed, 2).float()
    return x.to(xd), res, w.to(wd)


BF, F = torch.bfloat16, torch.float32
TYPES = [(BF, None, BF), (BF, BF, BF), (BF, F, F), (F, None, BF), (F, F, F), (BF, BF, F)]
SHAPES = [(1, 16), (5, 16), (3, 48), (67, 128), (2, 144), (33, 1024), (9, 1040), (4, 2064), (7, 5120), (2, 8192),
          (3, 16384)]


def _oracle(x, res, w, eps):
    return o.rmsnorm(_f(x), _f(w), eps, None if res is None else _f(res),
                     "f32" if res is not None and res.dtype == F else "bf16")


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("xd,rd,wd", TYPES)
def test_outputs_bitwise(m, k, xd, rd, wd):
    x, res, w = _inputs(m, k, xd, rd, wd, m + k)
    r_ref, y_ref = _oracle(x, res, w, 1e-6)
    xd_, wd_ = x.to(DEV), w.to(DEV)
    rd_ = None if res is None else res.to(DEV)
    got = nv().rmsnorm(xd_, wd_, 1e-6, rd_)
    y = got if res is None else got[0]
    assert y.dtype == BF and np.array_equal(_f(y), y_ref)
    if res is not None:
        assert got[1].dtype == rd and np.array_equal(_f(got[1]), r_ref)
    # the checkpoint form: the same y, and its packed form
    got = nv().rmsnorm_checkpoint(xd_, wd_, 1e-6, rd_)
    assert torch.equal(got[0], y)
    codes, scales = o.checkpoint_pack(y_ref)
    assert np.array_equal(got[-1].codes.cpu().numpy(), codes)
    assert np.array_equal(got[-1].scales.cpu().numpy(), scales)
    if res is not None:
        assert np.array_equal(_f(got[1]), r_ref)
    # NVFP4 codes, dynamic and static scale
    for gsf in (None, 3.5):
        got = nv().quantize_rmsnorm(xd_, wd_, 1e-6, rd_, gsf)
        g = o.global_sf(o.amax(y_ref)) if gsf is None else np.float32(gsf)
        packed, s8 = oracle_quantize(y_ref, g)
        assert np.float32(got[2].item()) == g
        assert np.array_equal(got[0].cpu().numpy(), packed)
        lay = got[1].cpu().numpy()
        assert np.array_equal(layout_to_canonical(lay, m, k), s8)
        kt = (k + 127) // 128
        assert not lay.reshape(kt, m, 8).transpose(1, 0, 2).reshape(m, -1)[:, k // 16:].any()   # padding bytes
        if res is not None:
            assert np.array_equal(_f(got[3]), r_ref)


@pytest.mark.parametrize("m,k", [(1, 5120), (2, 5120), (2, 16384), (3, 16384), (8, 16384), (9, 16384), (11, 144),
                                 (15, 8192), (16, 8192), (16, 8208), (17, 5120), (1025, 512), (4099, 512)])
def test_dynamic_equals_two_steps(m, k):
    """The one-row and the two-pass form (and past the row-walking grid): codes equal
    to quantizing the written norm."""
    x, res, w = (t.to(DEV) for t in _inputs(m, k, BF, BF, F, m))
    c, s, g, r = nv().quantize_rmsnorm(x, w, 1e-5, res)
    y, r2 = nv().rmsnorm(x, w, 1e-5, res)
    c2, s2, g2 = nv().quantize_activation(y)
    assert torch.equal(c, c2) and torch.equal(s, s2) and torch.equal(g, g2) and torch.equal(r, r2)


@pytest.mark.parametrize("m,k", [(1, 512), (6, 2048), (40, 1024)])
def test_residual_in_place(m, k):
    """The C call may update the residual (or x) in place, on every form."""
    from nvfp4_w4a4_quantized_global_amd._lib import check, lib
    x, res, w = (t.to(DEV) for t in _inputs(m, k, BF, BF, F, 5))
    c0, s0, g0, r0 = nv().quantize_rmsnorm(x, w, 1e-6, res)
    y0, _, ck0 = nv().rmsnorm_checkpoint(x, w, 1e-6, res)
    stream = torch.cuda.current_stream().cuda_stream
    for over in ("residual", "x"):
        for quantize in (True, False):
            xi, ri = x.clone(), res.clone()
            dst = ri if over == "residual" else xi
            args = (xi.data_ptr(), 0, ri.data_ptr(), 0, w.data_ptr(), 1, m, k, 1e-6)
            if quantize:
                c, s, g = torch.zeros_like(c0), torch.zeros_like(s0), torch.zeros_like(g0)
                need = lib().nvfp4_quantize_rmsnorm_workspace_bytes(m)
                ws = torch.empty((max(need, 1),), dtype=torch.uint8, device=DEV)
                check(lib().nvfp4_quantize_rmsnorm(*args, None, dst.data_ptr(), c.data_ptr(), s.data_ptr(), g.data_ptr(),
                                                   ws.data_ptr(), need, stream))
                assert torch.equal(c, c0) and torch.equal(s, s0) and torch.equal(g, g0)
            else:
                y, cc, cs = torch.empty_like(y0), torch.empty_like(ck0.codes), torch.empty_like(ck0.scales)
                check(lib().nvfp4_rmsnorm(*args, dst.data_ptr(), y.data_ptr(), cc.data_ptr(), cs.data_ptr(), stream))
                assert torch.equal(y, y0) and torch.equal(cc, ck0.codes) and torch.equal(cs, ck0.scales)
            assert torch.equal(dst, r0)


def test_accuracy_against_float64():
    x, res, w = _inputs(64, 5120, BF, F, F)
    y = _f(nv().rmsnorm(x.to(DEV), w.to(DEV), 1e-6, res.to(DEV))[0]).astype(np.float64)
    r = (_f(x) + _f(res)).astype(np.float64)
    ref = r / np.sqrt(np.mean(r * r, -1, keepdims=True) + np.float64(np.float32(1e-6))) * _f(w).astype(np.float64)
    # three fp32 roundings (the scale, two products), one to bf16
    assert np.all(np.abs(y - ref) <= np.abs(ref) * (2.0 ** -8 + 4 * U) + 2.0 ** -134)


def test_non_finite_rows_stay_theirs():
    x, _, w = _inputs(8, 256, BF, None, F)
    x[4, 7], x[5, 9] = float("inf"), float("nan")
    y = nv().rmsnorm(x.to(DEV), w.to(DEV))
    x0 = x.clone()
    x0[4, 7] = x0[5, 9] = 1.0
    y0 = nv().rmsnorm(x0.to(DEV), w.to(DEV))
    keep = [0, 1, 2, 3, 6, 7]
    assert torch.equal(y[keep], y0[keep])
    assert y[5].isnan().all() and y[4, 7].isnan()


def test_strided_misaligned_and_leading_dims():
    x, res, w = _inputs(6, 256, BF, BF, F)
    x, res, w = x.to(DEV), res.to(DEV), w.to(DEV)
    y, r = nv().rmsnorm(x, w, 1e-6, res)
    wide = torch.zeros((6, 300), dtype=BF, device=DEV)
    wide[:, 3:259] = x
    flat = torch.zeros(6 * 256 + 1, dtype=BF, device=DEV)
    flat[1:] = res.reshape(-1)
    y2, r2 = nv().rmsnorm(wide[:, 3:259], w, 1e-6, flat[1:].view(6, 256))
    assert torch.equal(y, y2) and torch.equal(r, r2)
    y3, r3 = nv().rmsnorm(x.view(2, 3, 256), w, 1e-6, res.view(2, 3, 256))
    assert y3.shape == (2, 3, 256) and torch.equal(y3.view(6, 256), y) and torch.equal(r3.view(6, 256), r)
    w2 = torch.zeros(257, device=DEV)
    w2[1:] = w
    assert torch.equal(nv().rmsnorm(x, w2[1:]), nv().rmsnorm(x, w))


def test_empty_input():
    x, w = torch.empty((0, 64), dtype=BF, device=DEV), torch.ones(64, device=DEV)
    assert nv().rmsnorm(x, w).shape == (0, 64)
    y, r, ck = nv().rmsnorm_checkpoint(x, w, 1e-6, x)
    assert ck.codes.shape == (0, 64) and ck.scales.shape == (0, 2) and r.shape == (0, 64)
    c, s, g = nv().quantize_rmsnorm(x, w)
    assert c.shape == (0, 32) and s.numel() == 0
    assert np.float32(g.item()) == o.global_sf(0.0) and nv().quantize_rmsnorm(x, w, 1e-6, x, 3.0)[2].item() == 3.0
    gx, gw = nv().rmsnorm_backward(x, x, w)
    assert gx.shape == (0, 64) and torch.equal(gw, torch.zeros_like(gw))


def _backward_bounds(gy, r, w, eps, gres, rows):
    gy, r, w = (np.asarray(a, dtype=np.float64) for a in (gy, r, w))
    k = r.shape[1]
    s = 1.0 / np.sqrt(np.mean(r * r, -1, keepdims=True) + np.float64(np.float32(eps)))
    n = np.abs(r) * s
    g = np.abs(gy * w)
    d = np.sum(np.abs(gy * w * r), -1, keepdims=True)       # 40 roundings at most on the way of a term of d
    q = 0.0 if gres is None else np.abs(np.asarray(gres, dtype=np.float64))
    tol_r = U * (8 * (s * g + q) + 50 * n * s * s * d / k)
    tol_w = U * (rows + 4) * np.sum(np.abs(gy) * n, 0)      # any order of the row sum
    return tol_r, tol_w


@pytest.mark.parametrize("rd,wd,with_res", [(BF, F, True), (BF, BF, False), (F, F, True), (F, BF, False)])
@pytest.mark.parametrize("m,k", [(1, 16), (3, 48), (70, 128), (2050, 160), (33, 1024), (9, 1040), (1100, 2064),
                                 (7, 5120), (3, 16384)])
def test_backward_against_formula(m, k, rd, wd, with_res):
    r, _, w = _inputs(m, k, rd, None, wd, m)
    if m > 3:
        r[1], r[2], r[3] = 1.0, 2.0, -3.0      # the fp32 gradient of extreme rows leaves fp32's range
    gy = workloads.draw("normal", (m, k), 71, 0, 1e-2)
    gres = workloads.draw("normal", (m, k), 72, 0, 1e-2).to(rd) if with_res else None
    gx, gw = nv().rmsnorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), 1e-6, None if gres is None else gres.to(DEV))
    assert gx.dtype == rd and gw.dtype == F
    ref_x, ref_w = o.rmsnorm_grads(_f(gy), _f(r), _f(w), 1e-6, None if gres is None else _f(gres))
    tol_r, tol_w = _backward_bounds(_f(gy), _f(r), _f(w), 1e-6, None if gres is None else _f(gres), m)
    if rd == BF:
        tol_r = tol_r + 2.0 ** -8 * (np.abs(ref_x) + tol_r)
    assert np.all(np.abs(_f(gx) - ref_x) <= tol_r + 2.0 ** -134)
    assert np.all(np.abs(_f(gw) - ref_w) <= tol_w + 2.0 ** -134)
    gx2, gw2 = nv().rmsnorm_backward(gy.to(DEV), r.to(DEV), w.to(DEV), 1e-6, None if gres is None else gres.to(DEV))
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)


def test_backward_zero_row():
    """A zero row: s = 1 / sqrt(eps), the gradient s g."""
    r = torch.zeros((2, 64), device=DEV)
    gy, w = torch.ones((2, 64), dtype=BF, device=DEV), torch.ones(64, device=DEV)
    gx, gw = nv().rmsnorm_backward(gy, r, w, 1e-4)
    s = 1.0 / np.sqrt(np.float64(np.float32(1e-4)))
    assert np.all(np.abs(_f(gx) - s) <= 4 * U * s) and not gw.any()


@pytest.mark.parametrize("rd", [None, BF, F])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_train_gradients(rd, checkpoint):
    """Through autograd: x, weight and residual all receive the formula's gradients; the
    residual output's own gradient joins in."""
    m, k = 37, 512
    x, res, w = _inputs(m, k, BF, rd, F, 9)
    x[2:4] = 1.5
    leaf = lambda t: None if t is None else t.to(DEV).requires_grad_(True)  # noqa: E731
    xl, rl, wl = leaf(x), leaf(res), leaf(w)
    out = nv().rmsnorm_train(xl, wl, 1e-6, rl, checkpoint)
    out = out if isinstance(out, tuple) else (out,)
    gy = workloads.draw("normal", (m, k), 73, 0, 1e-2).to(DEV)
    outs, grads = [out[0]], [gy]
    gr = None
    if rd is not None:
        gr = workloads.draw("normal", (m, k), 74, 0, 1e-2).to(DEV).to(rd)
        outs.append(out[1])
        grads.append(gr)
    if checkpoint:
        assert np.array_equal(out[-1].codes.cpu().numpy(), o.checkpoint_pack(_f(out[0]))[0])
        assert not out[-1].codes.requires_grad
    torch.autograd.backward(outs, grads)
    r = out[1].detach() if rd is not None else x.to(DEV)
    gx, gw = nv().rmsnorm_backward(gy, r, wl.detach(), 1e-6, gr)
    assert torch.equal(xl.grad, gx.to(BF)) and torch.equal(wl.grad, gw)
    if rd is not None:
        assert torch.equal(rl.grad, gx) and rl.grad.dtype == rd


def test_train_unused_outputs():
    """Only y, or only the residual stream, enters the loss."""
    x, res, w = (t.to(DEV) for t in _inputs(5, 64, BF, F, F, 1))
    x.requires_grad_(True), res.requires_grad_(True), w.requires_grad_(True)
    y, r = nv().rmsnorm_train(x, w, 1e-6, res)
    y.float().sum().backward()
    assert res.grad is not None and w.grad is not None
    x.grad = res.grad = w.grad = None
    y, r = nv().rmsnorm_train(x, w, 1e-6, res)
    r.sum().backward()
    assert torch.equal(res.grad, torch.ones_like(res)) and torch.equal(x.grad, torch.ones_like(x)) and w.grad is None


def test_train_against_differences():
    """d loss along random directions of x and w, loss = <y, gy> in float64 on the oracle's
    unrounded norm: the GPU gradient is the derivative (fp32 stream, so only y rounds)."""
    m, k = 4, 128
    g = np.random.default_rng(8)
    x, w = g.standard_normal((m, k)).astype(np.float32), (1 + 0.1 * g.standard_normal(k)).astype(np.float32)
    gy = torch.from_numpy(g.standard_normal((m, k))).to(BF)
    xl = torch.from_numpy(x).to(DEV).requires_grad_(True)
    wl = torch.from_numpy(w).to(DEV).requires_grad_(True)
    nv().rmsnorm_train(xl, wl, 1e-5).backward(gy.to(DEV))

    def loss(x, w):
        return np.sum(_f(gy) * x * w / np.sqrt(np.mean(x * x, -1, keepdims=True) + np.float64(np.float32(1e-5))))

    dx, dw, h = g.standard_normal((m, k)), g.standard_normal(k), 1e-5
    num = (loss(x + h * dx, w + h * dw) - loss(x - h * dx, w - h * dw)) / (2 * h)
    ana = np.sum(_f(xl.grad).astype(np.float64) * dx) + np.sum(_f(wl.grad).astype(np.float64) * dw)
    scale = np.sum(np.abs(_f(xl.grad) * dx)) + np.sum(np.abs(_f(wl.grad) * dw))
    assert abs(num - ana) <= 64 * U * scale + 1e-7 * scale      # fp32 gradients; differences to h^2


def test_refusals():
    lib = nv()
    x, w = torch.ones((4, 64), dtype=BF, device=DEV), torch.ones(64, device=DEV)
    for bad in (lambda: lib.rmsnorm(x[:, :24].contiguous(), w[:24]), lambda: lib.rmsnorm(x, w[:32]),
                lambda: lib.rmsnorm(x.half(), w), lambda: lib.rmsnorm(x, w.double()),
                lambda: lib.rmsnorm(x, w, 1e-6, x[:2]), lambda: lib.rmsnorm(x.float(), w, 1e-6, x),
                lambda: lib.rmsnorm(x, w, -1.0), lambda: lib.rmsnorm(x, w, float("nan")),
                lambda: lib.rmsnorm(x.cpu(), w), lambda: lib.rmsnorm(x, w.cpu()),
                lambda: lib.rmsnorm(x, w, 1e-6, x.cpu()),
                lambda: lib.rmsnorm(torch.ones((1, 16400), dtype=BF, device=DEV), torch.ones(16400, device=DEV)),
                lambda: lib.rmsnorm_backward(x, x[:2], w), lambda: lib.rmsnorm_backward(x, x, w, 1e-6, x.float()),
                lambda: lib.rmsnorm_backward(x.float(), x, w)):
        with pytest.raises(ValueError):
            bad()


def test_side_stream_and_graph_replays():
    """All forms captured on a side stream; each replay equals the eager calls on new inputs."""
    lib = nv()
    m, k = 130, 1280
    x, res, w = (t.to(DEV) for t in _inputs(m, k, BF, BF, F, 4))
    gy = workloads.draw("normal", (m, k), 75, 0, 1e-2).to(DEV)

    def call():
        return (*lib.quantize_rmsnorm(x, w, 1e-6, res), *lib.rmsnorm_checkpoint(x, w, 1e-6, res)[:2],
                *lib.rmsnorm_backward(gy, x, w, 1e-6, res), lib.quantize_rmsnorm(x[:1], w)[0])

    call()
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            out = call()
    torch.cuda.synchronize()
    for i in range(3):
        x.copy_(workloads.draw("t3", (m, k), 80 + i, 0).to(DEV))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        ref = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), f"replay {i}"


def test_two_streams_at_once():
    """Calls that overlap on two streams share nothing."""
    lib = nv()
    a, b = (tuple(t.to(DEV) for t in _inputs(257, 2048, BF, BF, F, 20 + i)) for i in range(2))
    ref = [lib.quantize_rmsnorm(x, w, 1e-6, res) for x, res, w in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, (x, res, w) in enumerate((a, b)):
            with torch.cuda.stream(s[i]):
                got[i] = lib.quantize_rmsnorm(x, w, 1e-6, res)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(got[i], ref[i]))
