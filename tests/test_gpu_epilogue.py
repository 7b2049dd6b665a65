"""The linear's epilogue with activation, residual and the stored pre-activation, on every
kernel path: out = bf16(act(z) + residual) from z = product + bias in fp32, one rounding.
References come from the plain linear (whose output is z rounded to bf16) and from the
float64 product of the dequantized operands; the training form's gradients follow the formula."""
import numpy as np
import pytest
import torch

import oracle as o
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


def _f(t):
    return t.detach().float().cpu().numpy()


# m, k, n, static scale: the paths by shape (one-row single launch plain and split, long
# row, fp16-activation decode, decode, skinny 2/4, pipelined 128-row, split tail, whole
# tiles; K % 32 != 0 takes the generic kernel; odd widths)
PATHS = [(1, 512, 96, None), (1, 5120, 1024, 8.0), (1, 25600, 400, None), (3, 1024, 333, None), (16, 1024, 1000, None),
         (20, 512, 96, 4.0), (40, 2048, 520, None), (100, 1024, 777, None), (300, 1280, 640, None), (513, 256, 257, None),
         (9, 272, 77, None), (300, 144, 300, None), (257, 528, 1024, 8.0),
         (100, 256, 4100, None), (128, 128, 4096, 4.0)]


def _case(m, k, n, gsf, seed=0):
    x = workloads.draw("normal", (m, k), 90 + seed, m).to(DEV)
    w = workloads.draw("normal", (n, k), 91 + seed, n, 0.05).to(DEV)
    b = workloads.draw("normal", (n,), 92 + seed, n, 0.5).to(DEV)
    res = workloads.draw("t3", (m, n), 93 + seed, m).to(DEV)
    g = None if gsf is None else torch.tensor(gsf, dtype=torch.float32, device=DEV)
    return x, nv().quantize_weight(w), b, res, g


def _plain(x, pk, sc, gw, b, n, g, *args, fn=None):
    """The plain linear's output without and with the bias."""
    fn = fn or nv().nvfp4_linear
    return fn(x, pk, sc, gw, None, n, g, *args), fn(x, pk, sc, gw, b, n, g, *args)


def _check(got, pre, plain, bias, act, res):
    """z lies within the plain linear's roundings: 2^-8 |y| of the product's and, with a bias,
    2^-8 of the sum's.  act is 1.13-Lipschitz; in fp32 its exponential's argument t rounds to
    2^-24 of itself and the rest are a handful of operations."""
    y, z0 = (_f(t).astype(np.float64) for t in plain)
    z = y if bias is None else z0
    dz = 2.0 ** -8 * np.abs(y) if bias is None else 2.0 ** -8 * (np.abs(y) + np.abs(z0) * 1.01)
    if pre is not None:
        if bias is None:
            assert torch.equal(pre, plain[0])
        else:
            assert np.all(np.abs(_f(pre) - z0) <= dz + 2.0 ** -8 * np.abs(z0) * 1.01 + 1e-30)
    v = o.activation(z, act)
    t = {"silu": np.abs(z), "gelu": z * z / 2, "gelu_tanh": 2 * np.abs(z) + np.abs(z) ** 3 / 10}.get(act, 0 * z)
    tol = 1.13 * dz * 1.01 + (np.minimum(t, 200) + 16) * 2.0 ** -22 * np.abs(v)
    if res is not None:
        v = v + _f(res).astype(np.float64)
    assert np.all(np.abs(_f(got) - v) <= 2.0 ** -8 * (np.abs(v) + tol) * 1.01 + tol + 1e-30)


@pytest.mark.parametrize("m,k,n,gsf", PATHS)
def test_every_path(m, k, n, gsf):
    lib = nv()
    x, (pk, sc, gw), b, res, g = _case(m, k, n, gsf)
    plain = _plain(x, pk, sc, gw, b, n, g)
    for bias in (None, b):
        pre = torch.empty((m, n), dtype=BF, device=DEV)
        for act, r in ((None, res), ("gelu", None), ("gelu_tanh", res), ("silu", res), (None, None)):
            pre.zero_()
            got = lib.nvfp4_linear(x, pk, sc, gw, bias, n, g, activation=act, residual=r, preact=pre)
            _check(got, pre, plain, bias, act, r)
            if act or r is not None:
                assert torch.equal(lib.nvfp4_linear(x, pk, sc, gw, bias, n, g, activation=act, residual=r), got)


@pytest.mark.parametrize("m,k,n", [(2048, 256, 8192), (2300, 128, 8200), (1100, 48, 6600)])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_whole_rounds_equal_row_slices(m, k, n, act):
    """At least one tile per compute unit (whole rounds; the fallback kernel's larger tile for
    K = 48): the same bits as 256-row slices of the call, under one static scale."""
    lib = nv()
    x, (pk, sc, gw), b, res, g = _case(m, k, n, 6.0)
    got = lib.nvfp4_linear(x, pk, sc, gw, b, n, g, activation=act, residual=res)
    for r in range(0, m, 256):
        part = lib.nvfp4_linear(x[r:r + 256], pk, sc, gw, b, n, g, activation=act, residual=res[r:r + 256])
        assert torch.equal(got[r:r + 256], part), r


@pytest.mark.parametrize("m,k,n", [(1, 512, 2048), (16, 1024, 1000), (40, 2048, 520), (300, 1280, 640), (300, 144, 300),
                                   (512, 256, 1024)])
@pytest.mark.parametrize("act", [None, "gelu", "gelu_tanh", "silu"])
def test_one_rounding_against_float64(m, k, n, act):
    """Every element within half a bf16 step (plus fp32's sum) of the float64 definition, and
    the error's norm that of one rounding: uniform within a step of 2^-7 |v| at most, its
    root mean square is at most 2^-7 / sqrt(12) = 0.00226 of the values'; a second rounding
    would add as much again."""
    lib = nv()
    x, (pk, sc, gw), b, res, _ = _case(m, k, n, None)
    res = res * 0.1
    c, s, g = lib.quantize_activation(x)
    one = torch.ones((), device=DEV)
    a, w = (lib.dequantize(*t, one, torch.float32).double() for t in ((c, s), (pk, sc)))
    alpha = float(np.float32(1.0) / np.float32(np.float32(g.item()) * np.float32(gw.item())))
    z = (a @ w.t().contiguous() * alpha + b.double()).cpu().numpy()
    bound = (a.abs() @ w.abs().t().contiguous() * alpha).cpu().numpy() * k * 2.0 ** -24
    got = _f(lib.nvfp4_linear(x, pk, sc, gw, b, n, activation=act, residual=res)).astype(np.float64)
    v = o.activation(z, act) + _f(res).astype(np.float64)
    tol = 1.13 * (bound + 2.0 ** -22 * np.abs(z)) + (np.minimum(z * z + 2 * np.abs(z) ** 3, 200) + 16) * 2.0 ** -22 * np.abs(z)
    assert np.all(np.abs(got - v) <= 2.0 ** -8 * np.abs(v) * 1.01 + tol + 1e-30)
    assert np.linalg.norm(got - v) <= (2.0 ** -7 / np.sqrt(12.0)) * np.linalg.norm(v)


@pytest.mark.parametrize("m,k,n,gsf", [(1, 512, 96, None), (16, 1024, 1000, None), (300, 1280, 641, None)])
def test_residual_updated_in_place(m, k, n, gsf):
    lib = nv()
    x, (pk, sc, gw), b, res, g = _case(m, k, n, gsf)
    ref = lib.nvfp4_linear(x, pk, sc, gw, b, n, g, activation="silu", residual=res)
    stream = res.clone()
    got = lib.nvfp4_linear(x, pk, sc, gw, b, n, g, out=stream, activation="silu", residual=stream)
    assert got.data_ptr() == stream.data_ptr() and torch.equal(stream, ref)


def test_misaligned_outputs_and_strided_residual():
    lib = nv()
    m, k, n = 130, 512, 264
    x, (pk, sc, gw), b, res, g = _case(m, k, n, None)
    ref = lib.nvfp4_linear(x, pk, sc, gw, b, n, g, activation="gelu_tanh", residual=res)
    flat = lambda: torch.empty(m * n + 1, dtype=BF, device=DEV)[1:].view(m, n)  # noqa: E731
    r1, out, pre = flat(), flat(), flat()
    r1.copy_(res)
    assert torch.equal(lib.nvfp4_linear(x, pk, sc, gw, b, n, g, out=out, activation="gelu_tanh", residual=r1, preact=pre), ref)
    _check(out, pre, _plain(x, pk, sc, gw, b, n, g), b, "gelu_tanh", res)
    wide = torch.zeros((m, n + 8), dtype=BF, device=DEV)
    wide[:, 8:] = res
    assert torch.equal(lib.nvfp4_linear(x, pk, sc, gw, b, n, g, activation="gelu_tanh", residual=wide[:, 8:]), ref)
    assert torch.equal(lib.nvfp4_linear(x.view(2, 65, k), pk, sc, gw, b, n, g, activation="gelu_tanh",
                                        residual=res.view(2, 65, n)).view(m, n), ref)


def test_rotation_swiglu_gemm_and_layer():
    lib = nv()
    m, k, n = 37, 1024, 256
    x, (pk, sc, gw), b, res, _ = _case(m, k, n, None)
    plain = _plain(x, pk, sc, gw, b, n, None, 16)
    _check(lib.nvfp4_linear(x, pk, sc, gw, b, n, None, 16, activation="silu", residual=res), None, plain, b, "silu", res)
    up = workloads.draw("normal", (m, k), 95, 0).to(DEV)
    for g in (None, torch.tensor(4.0, device=DEV)):
        plain = tuple(lib.nvfp4_linear_swiglu(x, up, pk, sc, gw, bias, n, g) for bias in (None, b))
        for act in (None, "gelu"):
            pre = torch.empty((m, n), dtype=BF, device=DEV)
            got = lib.nvfp4_linear_swiglu(x, up, pk, sc, gw, b, n, g, activation=act, residual=res, preact=pre)
            _check(got, pre, plain, b, act, res)
    c, s, g = lib.quantize_activation(x)
    plain = tuple(lib.nvfp4_gemm(c, s, pk, sc, g, gw, bias) for bias in (None, b))
    pre = torch.empty((m, n), dtype=BF, device=DEV)
    _check(lib.nvfp4_gemm(c, s, pk, sc, g, gw, b, activation="gelu_tanh", residual=res, preact=pre), pre, plain, b,
           "gelu_tanh", res)
    w = workloads.draw("normal", (n, k), 96, 0, 0.05).to(DEV)
    layer, bare = (lib.NVFP4Linear.from_weight(w, bias, 16) for bias in (b, None))
    _check(layer(x, "silu", res), None, (bare(x), layer(x)), b, "silu", res)


def test_non_finite_residual_stays_in_place():
    lib = nv()
    x, (pk, sc, gw), b, res, g = _case(20, 512, 96, None)
    ref = lib.nvfp4_linear(x, pk, sc, gw, b, 96, g, residual=res)
    res[3, 5], res[4, 6] = float("inf"), float("nan")
    got = lib.nvfp4_linear(x, pk, sc, gw, b, 96, g, residual=res)
    assert torch.isinf(got[3, 5]) and torch.isnan(got[4, 6])
    got[3, 5], got[4, 6] = ref[3, 5], ref[4, 6]
    assert torch.equal(got, ref)


def test_empty():
    lib = nv()
    x, (pk, sc, gw), b, res, g = _case(1, 512, 96, None)
    assert lib.nvfp4_linear(x[:0], pk, sc, gw, b, 96, g, activation="gelu", residual=res[:0]).shape == (0, 96)


def test_refusals():
    lib = nv()
    m, n = 4, 96
    x, (pk, sc, gw), b, res, g = _case(m, 512, n, None)
    buf = torch.empty(2 * m * n, dtype=BF, device=DEV)
    a, c = buf[:m * n].view(m, n), buf[8:m * n + 8].view(m, n)
    for kw in ({"activation": "relu"}, {"residual": res.float()}, {"residual": res[:2]}, {"residual": res.view(n, m)},
               {"residual": res.cpu()}, {"preact": torch.empty((m, n), device=DEV)},
               {"preact": torch.empty((n, m), dtype=BF, device=DEV)}, {"residual": a, "out": c}, {"residual": a, "preact": a},
               {"preact": a, "out": a}, {"residual": res, "out": torch.empty((n, m), dtype=BF, device=DEV)},
               {"residual": res, "workspace": torch.empty(1 << 20, dtype=torch.uint8)}):
        with pytest.raises(ValueError):
            lib.nvfp4_linear(x, pk, sc, gw, b, n, g, **kw)


def test_refuses_an_output_over_its_input():
    """Workgroups of one launch read the input while others write: h = linear(h) + h in place
    is refused, also where the ranges only touch at an end; next to it is fine."""
    lib = nv()
    m, k = 3, 512
    x, (pk, sc, gw), b, res, _ = _case(m, k, k, None)
    buf = torch.empty(3 * m * k, dtype=BF, device=DEV)
    h = buf[m * k:2 * m * k].view(m, k)
    h.copy_(x)
    for bad in (h, buf[8:m * k + 8].view(m, k), buf[2 * m * k - 8:3 * m * k - 8].view(m, k)):
        with pytest.raises(ValueError):
            lib.nvfp4_linear(h, pk, sc, gw, b, k, out=bad, residual=res)
        with pytest.raises(ValueError):
            lib.nvfp4_linear(h, pk, sc, gw, b, k, preact=bad, activation="silu")
        with pytest.raises(ValueError):
            lib.nvfp4_linear_swiglu(x, h, pk, sc, gw, b, k, out=bad, residual=res)
    ref = lib.nvfp4_linear(x, pk, sc, gw, b, k, residual=res)
    assert torch.equal(lib.nvfp4_linear(h, pk, sc, gw, b, k, out=buf[:m * k].view(m, k), residual=res), ref)
    assert torch.equal(lib.nvfp4_linear(h, pk, sc, gw, b, k, residual=h), lib.nvfp4_linear(x, pk, sc, gw, b, k, residual=x))


@pytest.mark.parametrize("g", [0, 16])
@pytest.mark.parametrize("act,with_res", [(None, True), ("silu", False), ("gelu", True), ("gelu_tanh", False)])
@pytest.mark.parametrize("packed", [False, True])
def test_train(g, act, with_res, packed):
    """Gradients of the training form against the float64 formula at the kept values: the
    input's checkpoint for grad_w, the kept z for act'."""
    lib = nv()
    m, k, n = 96, 512, 320
    x0, gy = workloads.draw("t3", (m, k), 97, g).to(DEV), workloads.draw("normal", (m, n), 98, g).to(DEV)
    w = workloads.draw("normal", (n, k), 97, 1, 0.05).float().to(DEV).requires_grad_(True)
    b = workloads.draw("normal", (n,), 97, 2).float().to(DEV).requires_grad_(True)
    res = workloads.draw("normal", (m, n), 97, 3).to(DEV).requires_grad_(True) if with_res else None
    x = x0.clone().requires_grad_(True)
    y = lib.nvfp4_linear_train(x, w, b, None, g, checkpoint=packed, activation=act, residual=res)
    pk, sc, gw = lib.quantize_weight(w.detach().to(BF))
    pre = torch.empty((m, n), dtype=BF, device=DEV)
    ref_y = lib.nvfp4_linear(x0, pk, sc, gw, b.detach().to(BF), n, None, g, activation=act,
                             residual=None if res is None else res.detach(), preact=pre)
    assert torch.equal(y.detach(), ref_y)
    y.backward(gy)
    kept = lib.checkpoint_pack(pre).dequantized() if packed else pre
    gz = torch.from_numpy(_f(gy) * o.activation_grad(_f(kept), act)).double()
    xr = o.rotate_activation(_f(x0), g, out="bf16") if g else _f(x0)
    if packed:
        xr = o.checkpoint_unpack(*o.checkpoint_pack(xr))
    xr = torch.from_numpy(np.asarray(xr, dtype=np.float64))
    # gz is rounded to bf16 (2^-8 of each term), then exact products and fp32 sums
    rel = (2.0 ** -8 if act else 0.0) + (m + n + 64) * 2.0 ** -22
    ref_w = gz.T @ xr
    assert torch.all((w.grad.cpu() - ref_w).abs() <= rel * (gz.abs().T @ xr.abs()))
    assert torch.all((b.grad.cpu() - gz.sum(0)).abs() <= rel * gz.abs().sum(0))
    wd = w.detach().double().cpu()
    gxr, mag = gz @ wd, gz.abs() @ wd.abs()
    if g:
        h = torch.from_numpy(o.sylvester_hadamard(g).astype(np.float64)) / np.sqrt(g)
        gxr = (gxr.view(-1, g) @ h).view(m, k)
        mag = (mag.view(-1, g) @ h.abs()).view(m, k)
    assert torch.all((x.grad.double().cpu() - gxr).abs() <= rel * mag + 2.0 ** -8 * (gxr.abs() + rel * mag))
    if with_res:
        assert torch.equal(res.grad, gy)


def test_train_residual_of_another_shape():
    """A residual given as [rows, N] to a [batch, tokens, K] input gets its gradient as [rows, N]."""
    lib = nv()
    x = workloads.draw("normal", (2, 6, 64), 110, 0).to(DEV)
    w = workloads.draw("normal", (48, 64), 110, 1).float().to(DEV)
    res = workloads.draw("normal", (12, 48), 110, 2).to(DEV).requires_grad_(True)
    y = lib.nvfp4_linear_train(x, w, residual=res, checkpoint=True)
    assert y.shape == (2, 6, 48)
    y.sum().backward()                     # an expanded, strided gradient
    assert torch.equal(res.grad, torch.ones_like(res))


def test_train_shared_checkpoint_block():
    """A block as it is trained: norm with residual and one checkpoint for both projections,
    SwiGLU from 8 bits, down projection onto the residual stream.  Every leaf gets the
    gradient of the same block built from bf16-keeping calls, up to the checkpoints' 2^-4."""
    lib = nv()
    m, k, f = 64, 256, 512
    d = lambda shape, i, s=1.0: workloads.draw("normal", shape, 99, i, s).float().to(DEV)  # noqa: E731
    leaves0 = [d((m, k), 0), d((m, k), 1), 1 + d((k,), 2, 0.1), d((f, k), 3, 0.05), d((f, k), 4, 0.05), d((k, f), 5, 0.05)]

    def block(packed):
        x, h, nw, wg, wu, wd = leaves = [t.clone().requires_grad_(True) for t in leaves0]
        out = lib.rmsnorm_train(x.to(BF), nw, 1e-6, h.to(BF), packed)
        y, r, ck = out if packed else (*out, None)
        gate = lib.nvfp4_linear_train(y, wg, checkpoint=ck)
        up = lib.nvfp4_linear_train(y, wu, checkpoint=ck)
        o_ = lib.nvfp4_linear_train(lib.swiglu_train(gate, up, packed), wd, checkpoint=packed or None, residual=r)
        o_.backward(d((m, k), 6).to(BF))
        return o_.detach(), [t.grad for t in leaves]

    y0, g0 = block(False)
    y1, g1 = block(True)
    assert torch.equal(y0, y1)
    for a, b in zip(g0, g1):
        assert torch.isfinite(b).all()
        assert (a - b).norm() <= 2.0 ** -4 * a.norm() * 2     # at most two checkpoints on the way of a leaf


@pytest.mark.parametrize("kw", [{"checkpoint": True}, {"activation": "silu"}])
def test_train_second_derivative_is_refused(kw):
    """The gradients of the checkpoint and the activation have no derivatives of their own: a
    derivative through them raises instead of missing terms.  First derivatives under
    create_graph stay what they are."""
    lib = nv()
    x = workloads.draw("normal", (6, 64), 111, 0).to(DEV).requires_grad_(True)
    w = workloads.draw("normal", (48, 64), 111, 1).float().to(DEV).requires_grad_(True)
    ref = torch.autograd.grad(lib.nvfp4_linear_train(x, w, **kw).float().sum(), (x, w))
    got = torch.autograd.grad(lib.nvfp4_linear_train(x, w, **kw).float().sum(), (x, w), create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    with pytest.raises(RuntimeError):
        sum(t.float().square().sum() for t in got).backward()


def test_flat_out_of_the_linear():
    """An ``out`` of another shape and as many values comes back in the output's shape."""
    lib = nv()
    x, (pk, sc, gw), b, _, _ = _case(20, 256, 96, None)
    ref = lib.nvfp4_linear(x, pk, sc, gw, b, 96)
    out = torch.empty(20 * 96, dtype=BF, device=DEV)
    got = lib.nvfp4_linear(x, pk, sc, gw, b, 96, out=out)
    assert got.shape == (20, 96) and got.data_ptr() == out.data_ptr() and torch.equal(got, ref)


def test_train_block_graph_replays():
    """Forward and backward of a block from 8-bit checkpoints captured once and replayed on new
    values, each replay against the eager block on other leaves with the same values (its
    graph is gone when the capture runs)."""
    lib = nv()
    m, k, f = 48, 256, 512
    d = lambda shape, i, s=1.0: workloads.draw("normal", shape, 112, i, s).float().to(DEV)  # noqa: E731
    shapes = [(m, k), (m, k), (k,), (f, k), (f, k), (k, f)]

    def values(seed):
        return [d(s, 10 * seed + i, 0.05 if i > 2 else 1.0) for i, s in enumerate(shapes)], d((m, k), 10 * seed + 9).to(BF)

    def step(leaves, gy):
        x, h, nw, wg, wu, wd = leaves
        y, r, ck = lib.rmsnorm_train(x.to(BF), nw, 1e-6, h.to(BF), True)
        gate = lib.nvfp4_linear_train(y, wg, checkpoint=ck)
        up = lib.nvfp4_linear_train(y, wu, checkpoint=ck, activation="gelu")
        out = lib.nvfp4_linear_train(lib.swiglu_train(gate, up, True), wd, checkpoint=True, residual=r)
        return [out.detach(), *torch.autograd.grad(out, leaves, gy)]

    def eager(seed):
        leaves, gy = values(seed)
        return [t.clone() for t in step([t.requires_grad_(True) for t in leaves], gy)]

    refs = [eager(s) for s in range(4)]
    leaves, gy = values(0)
    static = [t.requires_grad_(True) for t in leaves]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static, gy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(static, gy)
    for s in (1, 2, 3, 0):
        new, g = values(s)
        with torch.no_grad():
            for a, b in zip(static, new):
                a.copy_(b)
            gy.copy_(g)
        graph.replay()
        torch.cuda.synchronize()
        # the output and w_down's gradient come from this library's kernels alone: the same bits;
        # the others pass grad_y W products of the platform library, fp32 sums in an order of
        # its choice, whose bf16 rounding may fall one way or the other
        assert torch.equal(got[0], refs[s][0]) and torch.equal(got[6], refs[s][6])
        for a, b in zip(got, refs[s]):
            assert (a.float() - b.float()).norm() <= 1e-3 * b.float().norm()


def test_train_checkpoint_mismatch():
    lib = nv()
    x = torch.ones((4, 64), dtype=BF, device=DEV)
    w = torch.ones((32, 64), device=DEV)
    for bad in (lib.checkpoint_pack(x[:2]), lib.checkpoint_pack(x, 16)):
        with pytest.raises(ValueError):
            lib.nvfp4_linear_train(x, w, checkpoint=bad)
    with pytest.raises(TypeError):
        lib.nvfp4_linear_train(x, w, checkpoint=x)


def test_inference_block_and_graph():
    """A decode block captured and replayed: norm with residual into codes, two projections,
    SwiGLU into the down projection onto the stream in place, against eager calls."""
    lib = nv()
    k, f = 512, 1024
    ws = [lib.quantize_weight(workloads.draw("normal", s, 101, i, 0.05).to(DEV)) for i, s in enumerate(((f, k), (f, k), (k, f)))]
    nw = torch.ones(k, device=DEV)
    for m in (1, 7, 200):
        x, h = (torch.zeros((m, k), dtype=BF, device=DEV) for _ in range(2))

        def call(h):
            c, s, g, r = lib.quantize_rmsnorm(x, nw, 1e-6, h)
            gate, up = (lib.nvfp4_gemm(c, s, p, q, g, w) for p, q, w in ws[:2])
            p, q, w = ws[2]
            return lib.nvfp4_linear_swiglu(gate, up, p, q, w, None, k, out=r, residual=r)

        call(h)
        torch.cuda.synchronize()
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(st):
            with torch.cuda.graph(g, stream=st):
                out = call(h)
        torch.cuda.synchronize()
        for i in range(3):
            x.copy_(workloads.draw("normal", (m, k), 102 + i, m).to(DEV))
            h.copy_(workloads.draw("t3", (m, k), 105 + i, m).to(DEV))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            got = out.clone()
            ref = call(h)
            torch.cuda.synchronize()
            assert torch.equal(got, ref)
            y, r = lib.rmsnorm(x, nw, 1e-6, h)
            gate, up = (lib.nvfp4_linear(y, p, q, w, None, f) for p, q, w in ws[:2])
            p, q, w = ws[2]
            assert torch.equal(ref, lib.nvfp4_linear(lib.swiglu(gate, up), p, q, w, None, k, residual=r))
