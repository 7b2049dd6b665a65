"""The norm, epilogue and checkpoint operators on arrays of more than 2^31 values: an index
that wraps at 32 bits reads or writes the wrong rows.  Each of them treats its rows (or
values) independently, so the last rows of the large call equal a call on those rows alone,
bit for bit; the weight gradient is compared on small integers, whose sums are exact in any
order."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
LAST = 300


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


def _draw(rows, k, seed):
    """Normal values without a large fp32 copy: a block of rows, repeated under row factors."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    block = torch.randn((1000, k), generator=g, device=DEV).to(BF)
    x = torch.empty((rows, k), dtype=BF, device=DEV)
    for i in range(0, rows, 1000):
        x[i:i + 1000] = block[:min(1000, rows - i)] * (1 + i % 7)
    return x


@pytest.fixture(scope="module")
def tall():
    """More than 2^31 values: 131500 rows of 16384."""
    return _draw(131500, 16384, 1)


def test_norm_forms(tall):
    lib = nv()
    m, k = tall.shape
    assert m * k > 2 ** 31 + LAST * k
    w = torch.linspace(0.5, 1.5, k, device=DEV)
    tail = tall[-LAST:].clone()
    y, r, ck = lib.rmsnorm_checkpoint(tall, w, 1e-6, tall)
    y1, r1, ck1 = lib.rmsnorm_checkpoint(tail, w, 1e-6, tail)
    for a, b in ((y, y1), (r, r1), (ck.codes, ck1.codes), (ck.scales, ck1.scales)):
        assert torch.equal(a[-LAST:], b)
    del y, r, ck
    c, s, _ = lib.quantize_rmsnorm(tall, w, global_sf_x=20.0)
    c1, s1, _ = lib.quantize_rmsnorm(tail, w, global_sf_x=20.0)
    assert torch.equal(c[-LAST:], c1)
    assert torch.equal(s.view(k // 128, m, 8)[:, -LAST:], s1.view(k // 128, LAST, 8))
    c, _, g = lib.quantize_rmsnorm(tall, w)                       # dynamic: the same codes under its own scale
    assert torch.equal(c[-LAST:], lib.quantize_rmsnorm(tail, w, global_sf_x=g)[0])
    del c, s
    gr, gw = lib.rmsnorm_backward(tall, tall, w, 1e-6, tall)
    gr1, _ = lib.rmsnorm_backward(tail, tail, w, 1e-6, tail)
    assert torch.equal(gr[-LAST:], gr1) and torch.isfinite(gw).all()


def test_checkpoint_forms(tall):
    lib = nv()
    tail = tall[-LAST:].clone()
    ck, ck1 = lib.checkpoint_pack(tall, 16), lib.checkpoint_pack(tail, 16)
    assert torch.equal(ck.codes[-LAST:], ck1.codes) and torch.equal(ck.scales[-LAST:], ck1.scales)
    assert torch.equal(ck.dequantized()[-LAST:], ck1.dequantized())
    x, g, u = lib.swiglu_checkpoint(tall, tall)
    x1, g1, u1 = lib.swiglu_checkpoint(tail, tail)
    assert torch.equal(x[-LAST:], x1) and torch.equal(g.codes[-LAST:], g1.codes) and torch.equal(u.scales[-LAST:], u1.scales)
    dg, du = lib.swiglu_backward(tall, g, u)
    dg1, du1 = lib.swiglu_backward(tail, g1, u1)
    assert torch.equal(dg[-LAST:], dg1) and torch.equal(du[-LAST:], du1)
    for z, z1 in ((tall, tail), (g, g1)):
        assert torch.equal(lib.activation_backward(tall, z, "gelu")[-LAST:], lib.activation_backward(tail, z1, "gelu"))


def _integers(rows, k, seed, most):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-most, most + 1, (rows, k), generator=g, device=DEV, dtype=torch.int8).to(BF)


@pytest.mark.parametrize("act", ["gelu", None])
def test_linear_epilogue(act):
    """Operands of 6 and small integers: block scales are exact, the products' sums are integer
    multiples of 49 * 2^12 below 2^24 of them, exact in fp32 in any order, on every path."""
    lib = nv()
    m, k, n = 84300, 128, 25600
    assert m * n > 2 ** 31 + LAST * n
    x, w = _integers(m, k, 2, 3), _integers(n, k, 3, 3)
    x[:, ::16] = 6.0
    w[:, ::16] = 6.0
    pk, sc, gw = lib.quantize_weight(w)
    res = _draw(m, n, 4)
    bias = torch.linspace(-1, 1, n, device=DEV).to(BF)
    pre = torch.empty((m, n), dtype=BF, device=DEV)
    out = lib.nvfp4_linear(x, pk, sc, gw, bias, n, 448.0, activation=act, residual=res, preact=pre)
    pre1 = torch.empty((LAST, n), dtype=BF, device=DEV)
    tail = lib.nvfp4_linear(x[-LAST:].clone(), pk, sc, gw, bias, n, 448.0, activation=act, residual=res[-LAST:].clone(),
                            preact=pre1)
    assert torch.equal(out[-LAST:], tail) and torch.equal(pre[-LAST:], pre1)
    z = x[-LAST:].float() @ w.float().t() + bias.float()
    assert (pre1.float() - z).abs().max() <= (2.0 ** -8 + 2.0 ** -20) * z.abs().max()


@pytest.mark.parametrize("m,n,k", [(84300, 25600, 32), (1500, 4096, 4352), (1500, 4100, 4352), (5000, 136, 272), (320, 8192, 2064)])
def test_weight_grad_on_integers(m, n, k):
    """More than 2^31 gradient values, and both tile forms over many steps: integers up to 4
    and 3 sum to less than 2^24, exact in fp32 in any order, so the bits are known."""
    lib = nv()
    assert 12 * m < 2 ** 24
    gy, x = _integers(m, n, m + n, 4), _integers(m, k, m + k, 3)
    ref = torch.zeros((n, k), device=DEV)
    for i in range(0, m, 10000):
        ref += gy[i:i + 10000].float().t().contiguous() @ x[i:i + 10000].float()
    ck = lib.checkpoint_pack(x)
    assert torch.equal(ck.dequantized(), x)
    for _ in range(3):
        assert torch.equal(lib.weight_grad(gy, ck), ref)


@pytest.mark.parametrize("m,n,k", [(2, (1 << 24) + 8, 256), (3, (1 << 24) + 3, 16), (2, 24, (1 << 24) + 16)])
def test_weight_grad_widest(m, n, k):
    """Widths whose rows of a step pass 31-bit byte offsets, in both tile forms."""
    lib = nv()
    gy, x = _integers(m, n, 5, 4), _integers(m, k, 6, 3)
    got = lib.weight_grad(gy, lib.checkpoint_pack(x), BF)
    step = 1 << 20 if n > k else n
    for i in range(0, n, step):
        ref = gy[:, i:i + step].float().t().contiguous() @ x.float()      # at most 36: exact in bf16
        assert torch.equal(got[i:i + step].float(), ref)
