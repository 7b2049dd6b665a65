"""Outputs that a caller gives to the linears, on the GPU: refusals, and what lies behind a
larger buffer's part stays as it was."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _case(m, k, n):
    import nvfp4_w4a4_quantized_global_amd as nv
    x = workloads.draw("normal", (m, k), 230, m).to(DEV)
    return nv, x, nv.quantize_weight(workloads.draw("normal", (n, k), 231, n, 0.05).to(DEV))


@pytest.mark.parametrize("m", [1, 3, 20, 300])
def test_refused_without_an_epilogue(m):
    k, n = 256, 256
    nv, x, (pk, sc, gw) = _case(m, k, n)
    c, s, g = nv.quantize_activation(x)
    ref = nv.nvfp4_linear(x, pk, sc, gw, None, n)
    buf = torch.zeros((m + 1, n), dtype=BF, device=DEV)
    bad = (buf[:m - 1], buf.float()[:m], buf[:m].cpu(), torch.zeros((m, 2 * n), dtype=BF, device=DEV)[:, ::2], x)
    for out in bad:
        for call in (lambda: nv.nvfp4_linear(x, pk, sc, gw, None, n, out=out),
                     lambda: nv.nvfp4_linear_swiglu(x, x, pk, sc, gw, None, n, out=out),
                     lambda: nv.nvfp4_linear_segmented(x, 1, pk, sc, gw, None, n, out=out),
                     lambda: nv.nvfp4_linear_noalloc(x, pk, sc, gw, None, n, out=out)):
            with pytest.raises(ValueError):
                call()
        if out is not x:      # the product reads the codes
            with pytest.raises(ValueError):
                nv.nvfp4_gemm(c, s, pk, sc, g, gw, out=out)
    with pytest.raises(ValueError):
        nv.nvfp4_linear(x, pk, sc, gw, None, n, workspace=torch.zeros(1 << 24, dtype=torch.uint8))
    assert torch.equal(nv.nvfp4_linear(x, pk, sc, gw, None, n), ref)      # nothing is left behind
    buf[m:] = 7.0
    got = nv.nvfp4_gemm(c, s, pk, sc, g, gw, out=buf)
    assert got is buf and torch.equal(buf[:m], nv.nvfp4_gemm(c, s, pk, sc, g, gw)) and bool((buf[m:] == 7.0).all())


@pytest.mark.parametrize("m", [2, 20, 300])
def test_residual_stream_of_three_dimensions_in_place(m):
    """A [batch, tokens, N] stream updated in place, and preact of that shape."""
    k, n = 256, 136
    nv, x, (pk, sc, gw) = _case(m, k, n)
    h = workloads.draw("t3", (m, n), 232, m).to(DEV)
    ref_pre = torch.empty((m, n), dtype=BF, device=DEV)
    ref = nv.nvfp4_linear(x, pk, sc, gw, None, n, activation="gelu", residual=h, preact=ref_pre)
    stream, pre = h.clone().view(2, m // 2, n), torch.empty((2, m // 2, n), dtype=BF, device=DEV)
    got = nv.nvfp4_linear(x.view(2, m // 2, k), pk, sc, gw, None, n, activation="gelu", residual=stream, out=stream,
                          preact=pre)
    assert got.data_ptr() == stream.data_ptr() and got.shape == stream.shape
    assert torch.equal(stream.view(m, n), ref) and torch.equal(pre.view(m, n), ref_pre)
    down = nv.quantize_weight(workloads.draw("normal", (k, n - 8), 233, k, 0.05).to(DEV))
    g, u = (workloads.draw("normal", (m, n - 8), 234, i).to(DEV) for i in range(2))
    stream = workloads.draw("t3", (m, k), 235, m).to(DEV)
    ref = nv.nvfp4_linear_swiglu(g, u, *down, None, k, residual=stream)
    s3 = stream.view(2, m // 2, k)
    nv.nvfp4_linear_swiglu(g.view(2, m // 2, n - 8), u.view(2, m // 2, n - 8), *down, None, k, residual=s3, out=s3)
    assert torch.equal(stream, ref)


@pytest.mark.parametrize("kw", [{}, {"rotation_group": 16}, {"act_scale": "unit"}])
def test_layer_updates_its_stream_in_place(kw):
    """NVFP4Linear takes the epilogue's out and preact too."""
    import nvfp4_w4a4_quantized_global_amd as nv
    m, k, n = 12, 256, 128
    layer = nv.NVFP4Linear.from_weight(workloads.draw("normal", (n, k), 236, 0, 0.05).to(DEV),
                                       workloads.draw("normal", (n,), 236, 1).to(DEV), **kw)
    x = workloads.draw("normal", (2, m // 2, k), 237, 0).to(DEV)
    h = workloads.draw("t3", (2, m // 2, n), 237, 1).to(DEV)
    ref, z = layer(x, "silu", h), torch.empty_like(h)
    stream = h.clone()
    got = layer(x, activation="silu", residual=stream, out=stream, preact=z)
    assert got.data_ptr() == stream.data_ptr() and torch.equal(stream, ref)
    assert torch.equal(layer(x, residual=h), nv.nvfp4_linear(
        x, layer.packed, layer.inv_scale, layer.global_sf_w, layer.bias, n, layer.activation_global_sf(),
        layer.rotation_group or 0, residual=h))
    plain = torch.empty_like(h)
    assert torch.equal(layer(x, out=plain), layer(x)) and torch.equal(plain, layer(x))
    # z is the sum before the activation, rounded once: within the roundings of the plain linear's two
    y = layer(x).float()
    assert ((z.float() - y).abs() <= 2.0 ** -8 * (z.float().abs() + 3 * y.abs() + 2 * layer.bias.float().abs())).all()


def test_a_stream_that_the_norms_gradient_saved():
    """Updating in place the stream that rmsnorm_train saved is an error in its backward, not a
    gradient at the new values."""
    import nvfp4_w4a4_quantized_global_amd as nv
    m, k = 6, 256
    x = workloads.draw("normal", (m, k), 238, 0).to(DEV).requires_grad_(True)
    h = workloads.draw("t3", (m, k), 238, 1).to(DEV)
    wt = torch.ones(k, device=DEV)
    layer = nv.NVFP4Linear.from_weight(workloads.draw("normal", (k, k), 239, 0, 0.05).to(DEV))
    for update in (True, False):
        y, r = nv.rmsnorm_train(x, wt, 1e-6, h)
        stream = r.detach() if update else r.detach().clone()
        layer(y.detach(), residual=stream, out=stream)
        x.grad = None
        if update:
            with pytest.raises(RuntimeError, match="inplace"):
                y.float().sum().backward()
        else:
            y.float().sum().backward()
            assert torch.isfinite(x.grad).all()
