"""8-bit activation checkpoints: packing bit for bit against the oracle, and the gradients
computed from them (weight gradient, SwiGLU, activations) against float64 formulas at the
checkpoint's values."""
import numpy as np
import pytest
import torch

import oracle as o
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF = torch.bfloat16


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


def _f(t):
    return t.detach().float().cpu().numpy()


def _x(m, k, seed):
    """Heavy-tailed values; with room, a zero block, a huge and a tiny row, ties and edges of
    the format (448 and just above it times powers of two)."""
    x = workloads.draw("t3", (m, k), seed, 0).float()
    if m > 3:
        x[1] *= 1e30
        x[2] *= 1e-36
        x[3, :16] = 0.0
        x[3, 16:] = 0.0
    edge = torch.tensor([448.0, 450.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, -0.0], dtype=torch.float32)
    x[0, :8] = edge
    return x.to(BF)


@pytest.mark.parametrize("m,k", [(1, 16), (5, 48), (33, 128), (3, 144), (130, 1040), (2, 25600)])
def test_pack_bitwise(m, k):
    x = _x(m, k, m + k)
    ck = nv().checkpoint_pack(x.to(DEV))
    codes, scales = o.checkpoint_pack(_f(x))
    assert np.array_equal(ck.codes.cpu().numpy(), codes) and np.array_equal(ck.scales.cpu().numpy(), scales)
    ref = o.checkpoint_unpack(codes, scales)
    assert np.array_equal(ck.dequantized(torch.float32).cpu().numpy().astype(np.float64), ref)
    assert np.array_equal(_f(ck.dequantized()).astype(np.float64), ref)      # exact in bf16


@pytest.mark.parametrize("g", [2, 16, 128])
def test_pack_rotated(g):
    x = workloads.draw("t3", (37, 384), 5, g)
    ck = nv().checkpoint_pack(x.to(DEV), g)
    codes, scales = o.checkpoint_pack(o.rotate_activation(_f(x), g, out="bf16"))
    assert ck.rotation_group == g
    assert np.array_equal(ck.codes.cpu().numpy(), codes) and np.array_equal(ck.scales.cpu().numpy(), scales)


def test_pack_non_finite_and_leading_dims():
    x = _x(6, 64, 3)
    x[4, 3], x[4, 40], x[5, 63] = float("inf"), float("-inf"), float("nan")
    ck = nv().checkpoint_pack(x.to(DEV).view(2, 3, 64))
    assert ck.codes.shape == (2, 3, 64) and ck.scales.shape == (2, 3, 2)
    v = ck.dequantized().view(6, 64).float().cpu()
    ref = torch.from_numpy(o.checkpoint_unpack(*o.checkpoint_pack(_f(x)))).float()
    assert torch.equal(v.isnan(), ref.isnan()) and v.isnan().sum() == 3
    assert torch.equal(v.nan_to_num(), ref.nan_to_num())


WG = [(1, 16, 16), (4200, 136, 272), (140, 4096, 4112), (66, 4099, 4112), (1, 300, 272), (63, 8, 48), (64, 256, 256), (65, 264, 272), (777, 1024, 512), (130, 129, 144),
      (2000, 40, 5120), (513, 1000, 1040)]


@pytest.mark.parametrize("m,n,k", WG)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_weight_grad(m, n, k, dtype):
    x = workloads.draw("t3", (m, k), 31, m)
    gy = workloads.draw("normal", (m, n), 32, n, 1e-2)
    ck = nv().checkpoint_pack(x.to(DEV))
    got = nv().weight_grad(gy.to(DEV), ck, dtype)
    assert got.dtype == dtype and got.shape == (n, k)
    xv = o.checkpoint_unpack(ck.codes.cpu().numpy(), ck.scales.cpu().numpy())
    g = _f(gy).astype(np.float64)
    ref = g.T @ xv
    tol = (m + 2) * U * (np.abs(g).T @ np.abs(xv))           # fp32 sum of exact products, any order
    if dtype == BF:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(_f(got) - ref) <= tol + 1e-30)
    assert torch.equal(nv().weight_grad(gy.to(DEV), ck, dtype), got)


@pytest.mark.parametrize("m,n,k", [(1, 8, 16), (1, 9, 32), (1, 15, 16), (63, 9, 48), (64, 11, 32), (65, 9, 272), (129, 13, 16),
                                   (3, 5, 64), (200, 7, 48), (700, 251, 2064), (128, 2047, 5136), (3000, 61, 1024)])
def test_weight_grad_odd_widths_on_integers(m, n, k):
    """Rows of grad_y that start anywhere, the last of them ending inside a 16-byte load: small
    integers, whose sums are exact in any order.  Infinities reach their own output rows only:
    the first column's next row lies in the last load of each row."""
    g = torch.Generator().manual_seed(m + n + k)
    gy = torch.randint(-4, 5, (m, n), generator=g).to(BF).to(DEV)
    x = torch.randint(1, 4, (m, k), generator=g).to(BF).to(DEV)
    ck = nv().checkpoint_pack(x)
    ref = gy.double().t().contiguous() @ x.double()
    for dtype in (torch.float32, BF):
        assert torch.equal(nv().weight_grad(gy, ck, dtype), ref.float().to(dtype))
    gy[:, 0] = float("inf")
    got = nv().weight_grad(gy, ck)
    assert torch.isinf(got[0]).all() and torch.equal(got[1:], ref[1:].float())


def test_weight_grad_unsplit_equals_the_formula():
    """Without its workspace the C call runs unsplit."""
    import ctypes

    from nvfp4_w4a4_quantized_global_amd._lib import check, lib
    m, n, k = 1000, 256, 512
    x, gy = workloads.draw("normal", (m, k), 33, 0), workloads.draw("normal", (m, n), 34, 0).to(DEV)
    ck = nv().checkpoint_pack(x.to(DEV))
    assert lib().nvfp4_weight_grad_workspace_bytes(m, n, k) > 0
    out = torch.empty((n, k), device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    check(lib().nvfp4_weight_grad(p(gy), m, n, p(ck.codes), p(ck.scales), k, p(out), 1, None, 0,
                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    torch.cuda.synchronize()
    xv = o.checkpoint_unpack(ck.codes.cpu().numpy(), ck.scales.cpu().numpy())
    g = _f(gy).astype(np.float64)
    assert np.all(np.abs(_f(out) - g.T @ xv) <= (m + 2) * U * (np.abs(g).T @ np.abs(xv)))


def test_weight_grad_empty_and_non_finite():
    lib = nv()
    e = torch.empty((0, 64), dtype=BF, device=DEV)
    assert torch.equal(lib.weight_grad(e, lib.checkpoint_pack(e)), torch.zeros((64, 64), device=DEV))
    # an infinite gradient reaches its own output row only, as infinities of x's sign (rows
    # past the last one contribute nothing, not 0 * inf)
    m, n, k = 70, 24, 32
    x, gy = torch.ones((m, k), dtype=BF, device=DEV), torch.ones((m, n), dtype=BF, device=DEV)
    gy[m - 1, 5] = float("inf")
    got = lib.weight_grad(gy, lib.checkpoint_pack(x))
    assert torch.isinf(got[5]).all() and (got[5] > 0).all()
    keep = [i for i in range(n) if i != 5]
    assert torch.equal(got[keep], torch.full((n - 1, k), float(m), device=DEV))


def test_weight_grad_strided_gradient():
    m, n, k = 50, 48, 64
    wide = workloads.draw("normal", (m, 100), 35, 0).to(DEV)
    ck = nv().checkpoint_pack(workloads.draw("normal", (m, k), 36, 0).to(DEV))
    assert torch.equal(nv().weight_grad(wide[:, 3:51], ck), nv().weight_grad(wide[:, 3:51].contiguous(), ck))


def _silu_tol(gx, g, u):
    """fp32 sigmoid: its exponential's argument |g| rounds to 2^-24, exp2 and the reciprocal
    to an ulp, then a handful of products; relative to the terms' magnitudes."""
    sig = 1.0 / (1.0 + np.exp(-g))
    f = (np.abs(g) + 16) * 2.0 ** -22
    return f * np.abs(gx * u) * (sig + np.abs(g) * sig), f * np.abs(gx * g) * sig


@pytest.mark.parametrize("m,k", [(1, 16), (37, 272), (3, 25600), (260, 2048)])
@pytest.mark.parametrize("packed", [False, True])
def test_swiglu_forward_and_backward(m, k, packed):
    lib = nv()
    gate, up = workloads.draw("normal", (m, k), 41, 0, 3.0), workloads.draw("normal", (m, k), 41, 1, 3.0)
    gate.view(-1)[:6] = torch.tensor([0.0, 60.0, -60.0, 90.0, -90.0, 200.0]).to(BF)
    gx = workloads.draw("normal", (m, k), 41, 2)
    x, gc, uc = lib.swiglu_checkpoint(gate.to(DEV), up.to(DEV))
    assert torch.equal(x, lib.swiglu(gate.to(DEV), up.to(DEV)))
    for t, c in ((gate, gc), (up, uc)):
        codes, scales = o.checkpoint_pack(_f(t))
        assert np.array_equal(c.codes.cpu().numpy(), codes) and np.array_equal(c.scales.cpu().numpy(), scales)
    saved = (gc, uc) if packed else (gate.to(DEV), up.to(DEV))
    dg, du = lib.swiglu_backward(gx.to(DEV), *saved)
    gv, uv = (_f(t.dequantized() if packed else t).astype(np.float64) for t in saved)
    y = _f(gx).astype(np.float64)
    ref_g, ref_u = o.silu_grads(y, gv, uv)
    tol_g, tol_u = _silu_tol(y, gv, uv)
    assert np.all(np.abs(_f(dg) - ref_g) <= 2.0 ** -8 * (np.abs(ref_g) + tol_g) + tol_g + 1e-35)
    assert np.all(np.abs(_f(du) - ref_u) <= 2.0 ** -8 * (np.abs(ref_u) + tol_u) + tol_u + 1e-35)


@pytest.mark.parametrize("checkpoint", [False, True])
def test_swiglu_train(checkpoint):
    lib = nv()
    gate, up, gx = (workloads.draw("normal", (20, 96), 42, i).to(DEV) for i in range(3))
    g, u = gate.clone().requires_grad_(True), up.clone().requires_grad_(True)
    x = lib.swiglu_train(g, u, checkpoint)
    assert torch.equal(x.detach(), lib.swiglu(gate, up))
    x.backward(gx)
    saved = lib.swiglu_checkpoint(gate, up)[1:] if checkpoint else (gate, up)
    dg, du = lib.swiglu_backward(gx, *saved)
    assert torch.equal(g.grad, dg) and torch.equal(u.grad, du)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", None])
@pytest.mark.parametrize("m,n,packed", [(1, 1, False), (5, 37, False), (64, 256, False), (33, 272, True)])
def test_activation_backward(act, m, n, packed):
    lib = nv()
    z = workloads.draw("normal", (m, n), 43, n, 3.0)
    flat = z.view(-1)
    edge = torch.tensor([0.0, 12.0, -12.0, 95.0, -95.0, 3e38, -3e38, 1e-30]).to(BF)
    flat[: min(8, flat.numel())] = edge[: min(8, flat.numel())]
    gy = workloads.draw("normal", (m, n), 44, n)
    saved = lib.checkpoint_pack(z.to(DEV)) if packed else z.to(DEV)
    got = lib.activation_backward(gy.to(DEV), saved, act)
    zv = _f(saved.dequantized() if packed else saved).astype(np.float64)
    zc = np.clip(zv, -90, 90)                  # the derivative is 0 or 1 long before
    y = _f(gy).astype(np.float64)
    ref = y * o.activation_grad(zc, act)
    # The derivative is S + |z| S (1 - S) p' at most.  Its exponential's argument t rounds to
    # 2^-24 of itself, 1 - S to 2^-23 absolutely, times |z| p' <= 3 |t| + 2; the rest are a
    # handful of fp32 operations.
    p1 = np.sqrt(2 / np.pi)
    sig = lambda t: 1 / (1 + np.exp(-np.clip(t, -700, 700)))  # noqa: E731
    if act == "gelu":
        t = zc * zc / 2
        terms = np.abs(o.activation(zc, "gelu") / np.where(zc == 0, 1, zc)) + np.abs(zc) * np.exp(-t) / np.sqrt(2 * np.pi) + (zc == 0)
    elif act is None:
        t, terms = 0 * zc, 1 + 0 * zc
    else:
        t = np.abs(zc) if act == "silu" else 2 * p1 * np.abs(zc + 0.044715 * zc ** 3)
        dp = 1 if act == "silu" else 2 * p1 * (1 + 3 * 0.044715 * zc * zc)
        st = sig(np.sign(zc) * t)
        terms = st + np.abs(zc) * st * (1 - st) * dp
    tol = np.abs(y) * (3 * t + 16) * 2.0 ** -22 * terms
    assert np.all(np.abs(_f(got) - ref) <= 2.0 ** -8 * (np.abs(ref) + tol) + tol + 1e-35)


def test_activation_backward_nan():
    z = torch.full((1, 32), float("nan"), dtype=BF, device=DEV)
    for act in ("silu", "gelu", "gelu_tanh"):
        assert nv().activation_backward(torch.ones_like(z), z, act).isnan().all()


def test_refusals():
    lib = nv()
    x = torch.ones((4, 64), dtype=BF, device=DEV)
    ck = lib.checkpoint_pack(x)
    for bad in (lambda: lib.checkpoint_pack(x[:, :24].contiguous()), lambda: lib.checkpoint_pack(x.float()),
                lambda: lib.checkpoint_pack(x, 3), lambda: lib.checkpoint_pack(x, 256), lambda: lib.checkpoint_pack(x.cpu()),
                lambda: lib.checkpoint_unpack(ck, torch.float16),
                lambda: lib.checkpoint_unpack(lib.Checkpoint(ck.codes, ck.scales[:, :1])),
                lambda: lib.weight_grad(x[:2], ck), lambda: lib.weight_grad(x.float(), ck),
                lambda: lib.weight_grad(x, ck, torch.float16), lambda: lib.weight_grad(x, lib.Checkpoint(ck.codes, ck.scales.cpu())),
                lambda: lib.swiglu_backward(x, ck, x), lambda: lib.swiglu_backward(x, x[:2], x[:2]),
                lambda: lib.swiglu_backward(x, lib.checkpoint_pack(x, 16), ck),
                lambda: lib.activation_backward(x, x, "relu"), lambda: lib.activation_backward(x, x[:2], "silu"),
                lambda: lib.swiglu_checkpoint(x, x[:2])):
        with pytest.raises(ValueError):
            bad()


def test_graph_replays():
    lib = nv()
    m, n, k = 200, 264, 512
    x, gy = torch.empty((m, k), dtype=BF, device=DEV), torch.empty((m, n), dtype=BF, device=DEV)
    gx = workloads.draw("normal", (m, k), 45, 0).to(DEV)

    def call():
        ck = lib.checkpoint_pack(x, 16)
        y, g, u = lib.swiglu_checkpoint(x, gx)
        return (lib.weight_grad(gy, ck), ck.dequantized(), y, *lib.swiglu_backward(gx, g, u),
                lib.activation_backward(gx, lib.checkpoint_pack(x), "gelu"))

    x.fill_(1.0), gy.fill_(1.0)
    call()
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            out = call()
    torch.cuda.synchronize()
    for i in range(3):
        x.copy_(workloads.draw("t3", (m, k), 46 + i, 0).to(DEV))
        gy.copy_(workloads.draw("normal", (m, n), 46 + i, 1).to(DEV))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        ref = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), f"replay {i}"
