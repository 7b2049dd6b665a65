"""The 8-bit block-scaled linear: codes and scales bit for bit against the oracle, products against
the float64 product of the codes' values over every kernel path (streamed, few rows in one launch,
both tile sizes, tiles split along K), the epilogue, gradients, refusals, streams and graphs."""
import numpy as np
import pytest
import torch

import oracle as o
import workloads
from tests._util import bf16_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


def _f(t):
    return t.detach().float().cpu().numpy()


def _values(codes, scales, weight: bool):
    s = scales.cpu().numpy()
    return o.fp8_values(codes.cpu().numpy(), s if weight else s.T, 128 if weight else 1)


def _group_max(a):
    """Largest magnitude of every eight consecutive values of a row."""
    return torch.nn.functional.pad(a.abs(), (0, -a.shape[1] % 8)).reshape(a.shape[0], -1, 8).amax(-1)


def _product(a, b):
    """float64 product of values [M, K] and [N, K], and how far the kernels' may be from it.

    The matrix core adds products in groups of eight consecutive values of K: it aligns them to the
    group's largest exponent E and cuts each below 2^(E - 13) (seen by adding 2^16 and one small
    product: 2^3 arrives in the same group and 2^2 does not; in another group 2^-7 does).  2^E is at
    most the product of the group's largest magnitudes gx and gw, so a group loses at most
    8 2^-13 gx gw.  Groups and blocks are added in fp32, each step off by at most 2^-23 of sum |x w|,
    and scales round four times: (K + 4) 2^-23 sum |x w|."""
    bt = b.t().contiguous()
    bound = (a.shape[1] + 4) * 2.0 ** -23 * (a.abs() @ bt.abs()) + 2.0 ** -10 * (_group_max(a) @ _group_max(b).t().contiguous())
    return a @ bt, bound


def _check(got, xv, wv, bias=None, act=None, res=None, preact=None):
    """The product's bound, and 2^-23 of the sum with the bias.  The activations are 1.13-Lipschitz
    and off by a few units of 2^-22 of max(|z|, |act|); one rounding to bf16."""
    # on the GPU: numpy would take minutes
    z, dz = (t.cpu().numpy() for t in _product(*(torch.from_numpy(np.ascontiguousarray(t)).to(DEV) for t in (xv, wv))))
    if bias is not None:
        z = z + _f(bias)
        dz = dz + 2.0 ** -23 * np.abs(z)
    ref, d = z, dz
    if act is not None:
        ref = o.activation(z, act)
        d = 1.13 * dz + 2.0 ** -20 * np.maximum(np.abs(ref), np.minimum(np.abs(z), 1.0))
    if res is not None:
        ref = ref + _f(res).astype(np.float64).reshape(ref.shape)
    got = _f(got).astype(np.float64).reshape(ref.shape)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > d * 1.01 + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + 1e-37
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])
    if preact is not None:
        p = _f(preact).astype(np.float64).reshape(z.shape)
        assert np.all(np.abs(p - z) <= dz * 1.01 + 2.0 ** -8 * np.abs(z) * (1 + 2.0 ** -7) + 1e-37)


# ---- codes ----

def _rows(m, k, seed=0):
    x = workloads.draw("normal_outliers", (m, k), 200 + seed, m).float()
    if m > 2:
        x[1] = 0.0
        x[2] *= 1e-36
    if m > 3:
        x[3] *= 1e34
    if m > 4:
        x[4] = torch.linspace(-448, 448, k)       # every binade, ties among them
    return x


CODE_SHAPES = [(1, 16), (5, 16), (7, 128), (9, 144), (67, 1040), (33, 5120), (3, 16400), (300, 272)]


@pytest.mark.parametrize("m,k", CODE_SHAPES)
def test_activation_codes(m, k):
    x = _rows(m, k).to(BF)
    codes, scales = nv().fp8_quantize_activation(x.to(DEV))
    c, s = o.fp8_quantize(_f(x), 1)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s.T)
    # with column sums: the same codes; fp32 sums of m values
    again, s2, total = nv().fp8_quantize_activation(x.to(DEV), column_sum=True)
    assert torch.equal(again, codes) and torch.equal(s2, scales)
    x64 = _f(x).astype(np.float64)
    assert np.all(np.abs(_f(total) - x64.sum(0)) <= m * 2.0 ** -24 * np.abs(x64).sum(0))
    assert torch.equal(nv().fp8_quantize_activation(x.to(DEV), column_sum=True)[2], total)
    for dt in (F, BF):
        v = nv().fp8_dequantize(codes, scales, dt)
        want = torch.from_numpy(o.fp8_values(c, s, 1).astype(np.float32)).to(dt)
        assert v.dtype == dt and torch.equal(v.cpu(), want)


@pytest.mark.parametrize("m,k", CODE_SHAPES)
def test_codes_with_the_checkpoint(m, k):
    x = _rows(m, k, 5).to(BF).to(DEV)
    x[-1, ::7] = float("nan")
    x[-1, 3] = float("inf")
    codes, scales, ck = nv().fp8_quantize_checkpoint(x)
    want = nv().checkpoint_pack(x)
    assert torch.equal(ck.codes, want.codes) and torch.equal(ck.scales, want.scales) and ck.rotation_group == 0
    for got, ref in zip((codes, scales), nv().fp8_quantize_activation(x)):
        assert torch.equal(got, ref)
    assert nv().fp8_quantize_checkpoint(x.view(m, 1, k))[2].scales.shape == (m, 1, (k + 31) // 32)
    codes, scales, ck = nv().fp8_quantize_checkpoint(x[:0])
    assert codes.shape == (0, k) and ck.codes.shape == (0, k) and scales.shape[1] == 0


@pytest.mark.parametrize("m,k", [(1, 16), (5, 144), (67, 1040), (3, 25600)])
def test_swiglu_codes(m, k):
    g, u = (workloads.draw("normal", (m, k), 210 + i, m).to(DEV) for i in range(2))
    want = nv().fp8_quantize_activation(nv().swiglu(g, u))
    got = nv().fp8_quantize_swiglu(g, u)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n,k", [(1, 16), (16, 48), (100, 128), (128, 144), (129, 400), (304, 1040), (1001, 272)])
@pytest.mark.parametrize("dt", [BF, F])
def test_weight_codes(n, k, dt):
    w = (_rows(n, k, 3) * (1 + 2.0 ** -13)).to(dt)
    codes, scales = nv().fp8_quantize_weight(w.to(DEV))
    c, s = o.fp8_quantize(_f(w), 128)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    assert torch.equal(nv().fp8_dequantize(codes, scales, F).cpu(), torch.from_numpy(o.fp8_values(c, s, 128).astype(np.float32)))
    if n % 16 == 0:
        codes2, scales2, ct, st = nv().fp8_quantize_weight(w.to(DEV), transpose=True)
        assert torch.equal(codes2, codes) and torch.equal(scales2, scales)
        assert torch.equal(ct, codes.t()) and torch.equal(st, scales.t())


def test_special_values():
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(1))
    x[1, 3], x[1, 200], x[2, 5] = float("inf"), float("-inf"), float("nan")
    codes, scales = nv().fp8_quantize_activation(x.to(BF).to(DEV))
    c, s = o.fp8_quantize(_f(x.to(BF)), 1)
    nan = (c & 0x7F) == 0x7F
    got = codes.cpu().numpy()
    assert np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], c[~nan])
    assert np.array_equal(scales.cpu().numpy(), s.T)
    # a NaN reaches its row's outputs, and only those, streamed, in one launch and in tiles
    wc, ws = nv().fp8_quantize_weight(torch.randn(48, 256, device=DEV))
    for rows in (4, 40, 300):
        xr = x.to(BF).to(DEV).repeat(rows // 4 + 1, 1)[:rows]
        y = nv().fp8_linear(xr, wc, ws)
        bad = torch.tensor([r % 4 in (1, 2) for r in range(rows)], device=DEV)
        assert y[bad].isnan().all() and y[~bad].isfinite().all()


# ---- products ----

# m, k, n: few rows in one launch, streamed one to four activation tiles, small and large tiles,
# whole and split along K, ragged in every direction
PATHS = [(1, 16, 1), (1, 5120, 1024), (1, 25600, 400), (2, 144, 77), (4, 5120, 333), (4, 16384, 64), (5, 272, 1000),
         (16, 25600, 96), (17, 1040, 520), (33, 2064, 257), (64, 1024, 1001), (65, 5120, 1024), (100, 1040, 777),
         (130, 128, 136), (300, 1280, 640), (513, 272, 257), (257, 16, 300), (1000, 5120, 600), (129, 25600, 200)]


def _case(m, k, n, seed=0):
    x = workloads.draw("normal_outliers", (m, k), 220 + seed, m).to(DEV)
    w = workloads.draw("normal", (n, k), 221 + seed, n, 0.05)
    w[:, : k // 2] *= 8.0          # tiles of different scales
    b = workloads.draw("normal", (n,), 222 + seed, n, 0.5).to(DEV)
    res = workloads.draw("t3", (m, n), 223 + seed, m).to(DEV)
    return x, nv().fp8_quantize_weight(w.to(DEV)), b, res


# every count of activation and weight tiles of the streaming kernel (the weight's width decides the
# latter), rows that straddle the weight's scale blocks, quarter tiles after a whole round (some of
# them outside the output), two whole rounds, splits of quarter tiles
WIDTHS = [(1, 144, 5000), (3, 272, 9001), (16, 144, 5001), (9, 272, 12000), (20, 144, 300), (30, 144, 5000), (32, 272, 9000),
          (40, 144, 1000), (64, 144, 6000), (50, 272, 9003), (4100, 144, 5000), (4091, 272, 8200), (4352, 2064, 4096),
          (8300, 16, 8001)]


@pytest.mark.parametrize("m,k,n", PATHS + WIDTHS)
def test_linear(m, k, n):
    x, (wc, ws), b, res = _case(m, k, n)
    xc, xs = nv().fp8_quantize_activation(x)
    xv, wv = _values(xc, xs, False), _values(wc, ws, True)
    y = nv().fp8_linear(x, wc, ws)
    assert y.dtype == BF and y.shape == (m, n)
    _check(y, xv, wv)
    g = nv().fp8_gemm(xc, xs, wc, ws)
    _check(g, xv, wv)
    # the same inputs give the same bits; without a workspace for the splits the same function
    assert torch.equal(nv().fp8_linear(x, wc, ws), y)
    for act in ("gelu", "silu", "gelu_tanh") if m * n < 1 << 21 else ("silu",):
        pre = torch.empty(m, n, device=DEV, dtype=BF)
        _check(nv().fp8_linear(x, wc, ws, b, activation=act, residual=res, preact=pre), xv, wv, b, act, res, pre)
    _check(nv().fp8_gemm(xc, xs, wc, ws, b, residual=res), xv, wv, b, None, res)
    # in place on the residual stream
    h = res.clone()
    assert nv().fp8_linear(x, wc, ws, b, out=h, residual=h).data_ptr() == h.data_ptr()
    _check(h, xv, wv, b, None, res)


def test_block():
    """A pre-norm block as it is used: the norm writes codes, two projections read them, and the down
    projection of their SwiGLU product is added to the residual stream in place."""
    for m, k, f in [(1, 512, 1040), (7, 272, 528), (300, 512, 1040)]:
        x, h = workloads.draw("normal", (m, k), 260, m).to(DEV), workloads.draw("t3", (m, k), 261, m).to(DEV)
        lw, lb = (1 + 0.1 * torch.randn(k)).to(DEV), (0.1 * torch.randn(k)).to(DEV)
        gate, up, down = (nv().fp8_quantize_weight(0.05 * torch.randn(s, device=DEV)) for s in ((f, k), (f, k), (k, f)))
        for norm in ("layer", "rms"):
            if norm == "layer":
                codes, scales, r = nv().fp8_quantize_layernorm(x, lw, lb, 1e-6, h)
                y, r2 = nv().layernorm(x, lw, lb, 1e-6, h)
            else:
                codes, scales, r = nv().fp8_quantize_rmsnorm(x, lw, 1e-6, h)
                y, r2 = nv().rmsnorm(x, lw, 1e-6, h)
            assert torch.equal(r, r2)
            g, u = nv().fp8_gemm(codes, scales, *gate), nv().fp8_gemm(codes, scales, *up)
            yv = _values(*nv().fp8_quantize_activation(y), False)
            _check(g, yv, _values(*gate, True))
            _check(u, yv, _values(*up, True))
            out = nv().fp8_linear_swiglu(g, u, *down, out=r, residual=r)
            assert out.data_ptr() == r.data_ptr()
            p = nv().swiglu(g, u)
            _check(out, _values(*nv().fp8_quantize_activation(p), False), _values(*down, True), None, None, r2)
    # the same norm in front of 4-bit projections
    codes, scales, gsf = nv().quantize_layernorm(x, lw, lb)
    packed = nv().quantize_weight((0.05 * torch.randn(96, k, device=DEV)).to(BF))
    got = nv().nvfp4_gemm(codes, scales, packed[0], packed[1], gsf, packed[2])
    assert torch.equal(got, nv().nvfp4_linear(nv().layernorm(x, lw, lb), *packed, None, 96))


@pytest.mark.parametrize("m,k,n", [(1, 25600, 400), (3, 1040, 96), (16, 2064, 333), (300, 1280, 520)])
def test_linear_swiglu(m, k, n):
    g = workloads.draw("normal", (m, k), 230, m).to(DEV)
    x, (wc, ws), b, res = _case(m, k, n)
    want = nv().fp8_linear(nv().swiglu(g, x), wc, ws, b, residual=res)
    assert torch.equal(nv().fp8_linear_swiglu(g, x, wc, ws, b, residual=res), want)


def test_full_size_projections():
    # every projection of the decoder layer and the ViT block, at one row, 16, and an odd many
    for name, n, k in workloads.QWEN3_PROJECTIONS + workloads.VIT_LINEARS:
        w = torch.randn(n, k, device=DEV, dtype=F) * 0.02
        wc, ws = nv().fp8_quantize_weight(w)
        wv = nv().fp8_dequantize(wc, ws, F).double()
        for m in (1, 16, 777):
            x = torch.randn(m, k, device=DEV).to(BF)
            xv = nv().fp8_dequantize(*nv().fp8_quantize_activation(x), F).double()
            ref, bound = _product(xv, wv)
            bad = (nv().fp8_linear(x, wc, ws).double() - ref).abs() > bound * 1.01 + 2.0 ** -8 * 1.01 * ref.abs()
            assert not bad.any(), (name, m, int(bad.sum()))


def test_exact_integers():
    # codes of small integers under scales of one: sums below 2^24 are exact, whatever the path
    for m, k, n in [(1, 1024, 64), (20, 1024, 64), (300, 1024, 200), (700, 5120, 300)]:
        g = torch.Generator().manual_seed(m)
        x = torch.randint(-8, 9, (m, k), generator=g).float()
        w = torch.randint(-8, 9, (n, k), generator=g).float()
        xc, wc = (t.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV) for t in (x, w))
        xs = torch.ones((k + 127) // 128, m, device=DEV)
        ws = torch.ones((n + 127) // 128, (k + 127) // 128, device=DEV)
        want = (x.double() @ w.double().t()).float().to(BF)
        assert torch.equal(nv().fp8_gemm(xc, xs, wc, ws).cpu(), want)


def test_scales_reach_their_blocks():
    # one nonzero code per row and column block: every scale seen alone
    m, k, n = 300, 1040, 300
    xs = torch.rand((k + 127) // 128, m, device=DEV) + 0.5
    ws = torch.rand((n + 127) // 128, (k + 127) // 128, device=DEV) + 0.5
    one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    for blk in range((k + 127) // 128):
        xc, wc = torch.zeros(m, k, dtype=torch.uint8, device=DEV), torch.zeros(n, k, dtype=torch.uint8, device=DEV)
        xc[:, blk * 128 + 5] = wc[:, blk * 128 + 5] = one
        want = xs[blk][:, None].double() * ws[:, blk].repeat_interleave(128)[:n][None, :].double()
        for rows in (1, 3, 16, 40, 300):
            got = nv().fp8_gemm(xc[:rows].contiguous(), xs[:, :rows].contiguous(), wc, ws).double()
            assert ((got - want[:rows]).abs() <= (2.0 ** -8 + 2.0 ** -20) * want[:rows]).all(), (blk, rows)


def test_untouched_around_the_output():
    # rows and columns around a given output stay as they were
    for m, k, n in [(1, 272, 77), (20, 272, 77), (300, 272, 257)]:
        x, (wc, ws), b, _ = _case(m, k, n)
        buf = torch.full((m * n + 64,), 7.0, device=DEV, dtype=BF)
        out = buf[32:32 + m * n].view(m, n)
        assert torch.equal(nv().fp8_linear(x, wc, ws, b, out=out), nv().fp8_linear(x, wc, ws, b))
        assert (buf[:32] == 7).all() and (buf[32 + m * n:] == 7).all()
        odd = buf[1:1 + m * n].view(m, n)       # two-byte aligned
        assert torch.equal(nv().fp8_linear(x, wc, ws, b, out=odd), nv().fp8_linear(x, wc, ws, b))


@pytest.mark.parametrize("m,k,n", [(1, 272, 77), (20, 272, 77), (48, 1024, 528), (300, 1040, 528), (4096, 272, 2048)])
@pytest.mark.parametrize("act", [None, "gelu_tanh"])
def test_residual_in_place(m, k, n, act):
    # a residual stream updated where it lies, over every kind of kernel
    x, (wc, ws), b, res = _case(m, k, n)
    want = nv().fp8_linear(x, wc, ws, b, residual=res, activation=act)
    pre, want_pre = torch.empty_like(res), torch.empty_like(res)
    assert torch.equal(nv().fp8_linear(x, wc, ws, b, residual=res, activation=act, preact=want_pre), want)
    stream = res.clone()
    got = nv().fp8_linear(x, wc, ws, b, residual=stream, out=stream, activation=act, preact=pre)
    assert got.data_ptr() == stream.data_ptr() and torch.equal(stream, want) and torch.equal(pre, want_pre)


def test_long_offsets():
    # outputs and codes past 2^31
    m, k, n = 70000, 32, 32768
    x = torch.randn(64, k, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV).repeat(m // 64 + 1, 1)[:m]
    wc, ws = nv().fp8_quantize_weight(torch.randn(n, k, device=DEV))
    y = nv().fp8_linear(x, wc, ws)
    assert torch.equal(y[-48:], nv().fp8_linear(x[-48:].contiguous(), wc, ws))
    del y
    m, k, n = 140000, 16384, 48
    x = torch.randn(64, k, generator=torch.Generator().manual_seed(2)).to(BF).to(DEV).repeat(m // 64 + 1, 1)[:m]
    wc, ws = nv().fp8_quantize_weight(torch.randn(n, k, device=DEV) * 0.02)
    y, last = nv().fp8_linear(x, wc, ws), nv().fp8_linear(x[-200:].contiguous(), wc, ws)
    # another split of K: fp32 order
    assert ((y[-200:].float() - last.float()).abs() <= 2.0 ** -6 * last.float().abs() + 0.05).all()
    # a long row of one token
    k = 1 << 20
    x = torch.randn(1, k, device=DEV).to(BF)
    wc, ws = nv().fp8_quantize_weight(torch.randn(33, k, device=DEV) * 0.02)
    xv, wv = _values(*nv().fp8_quantize_activation(x), False), _values(wc, ws, True)
    _check(nv().fp8_linear(x, wc, ws), xv, wv)


def test_leading_dimensions_strides_and_empty():
    x, (wc, ws), b, res = _case(30, 144, 77)
    want = nv().fp8_linear(x, wc, ws, b, residual=res)
    x3 = x.view(5, 2, 3, 144)
    got = nv().fp8_linear(x3, wc, ws, b, residual=res.view(5, 2, 3, 77))
    assert got.shape == (5, 2, 3, 77) and torch.equal(got.view(30, 77), want)
    wide = torch.zeros(30, 300, device=DEV, dtype=BF)
    wide[:, 3:147] = x
    assert torch.equal(nv().fp8_linear(wide[:, 3:147], wc, ws, b, residual=res), want)
    assert torch.equal(nv().fp8_linear(x.t().contiguous().t(), wc, ws, b, residual=res), want)
    assert nv().fp8_linear(x[0], wc, ws).shape == (77,)
    assert nv().fp8_linear(x[:0], wc, ws).shape == (0, 77)
    assert nv().fp8_quantize_activation(x[:0])[1].shape == (2, 0)
    assert not nv().fp8_quantize_activation(x[:0], column_sum=True)[2].any()
    layer = nv().FP8Linear(wc, ws, b)
    assert torch.equal(layer(x, residual=res), want)
    w = workloads.draw("normal", (77, 144), 240, 1, 0.05).to(DEV)
    layer = nv().FP8Linear.from_weight(w.half(), b)
    assert layer(x).shape == (30, 77) and layer.dequantized_weight().shape == (77, 144)


def test_refusals():
    x, (wc, ws), b, res = _case(4, 144, 32)
    m, k, n = 4, 144, 32
    xc, xs = nv().fp8_quantize_activation(x)
    lin = nv().fp8_linear
    for bad in (lambda: lin(x[:, :128].contiguous(), wc, ws), lambda: lin(x.float(), wc, ws), lambda: lin(x, wc, ws[:, :1]),
                lambda: lin(x, wc, ws.t()), lambda: lin(x, wc.int(), ws), lambda: lin(x, wc, ws.double()),
                lambda: lin(x, wc, ws, b[:5]), lambda: lin(x, wc, ws, b.float()), lambda: lin(x, wc.cpu(), ws),
                lambda: lin(x, wc, ws, activation="relu"), lambda: lin(x, wc, ws, residual=res[:2]),
                lambda: lin(x, wc, ws, out=torch.empty(3, n, device=DEV, dtype=BF)),
                lambda: lin(x, wc, ws, out=torch.empty(m, n, device=DEV)),
                lambda: lin(x, wc, ws, preact=res, residual=res),
                lambda: lin(x[:, :8].contiguous(), wc[:, :8].contiguous(), ws[:, :1].contiguous()),
                lambda: nv().fp8_gemm(xc, xs.t().contiguous(), wc, ws), lambda: nv().fp8_gemm(xc[:, :128], xs, wc, ws),
                lambda: nv().fp8_quantize_weight(wc.half()), lambda: nv().fp8_quantize_weight(x[:, :20].contiguous()),
                lambda: nv().fp8_quantize_weight(torch.ones(20, 32, device=DEV), transpose=True),
                lambda: nv().fp8_dequantize(xc, xs[:, :2].contiguous()), lambda: nv().fp8_dequantize(xc, xs, torch.half),
                lambda: nv().fp8_linear_train(x, torch.ones(20, 144, device=DEV)),
                lambda: nv().fp8_linear_train(x, torch.ones(32, 128, device=DEV)),
                lambda: nv().fp8_linear_train(x, torch.ones(32, 144, device=DEV), checkpoint=nv().checkpoint_pack(x[:2])),
                lambda: nv().FP8Linear(wc, ws.t().contiguous()),
                lambda: nv().FP8Linear(wc.view(torch.float8_e4m3fnuz), ws), lambda: nv().FP8Linear(x[:, :80], ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        nv().fp8_linear_train(x, torch.ones(32, 144, device=DEV), checkpoint=True)
    xin = x.clone()
    with pytest.raises(ValueError):      # an output over the input
        nv().fp8_linear(xin[:, :32].contiguous().view(4, 32), *nv().fp8_quantize_weight(torch.ones(32, 32, device=DEV)),
                        out=xin.view(-1)[:128].view(4, 32), residual=xin.view(-1)[:128].view(4, 32), preact=xin.view(-1)[:128].view(4, 32))


# ---- training ----

def _train_reference(x, w, b, gy, act, res):
    """float64 gradients with the prescribed quantizations taken as given values."""
    xv = o.fp8_values(*o.fp8_quantize(_f(x), 1), 1)
    wv = o.fp8_values(*o.fp8_quantize(_f(w), 128), 128)
    return xv, wv


@pytest.mark.parametrize("m,k,n", [(1, 16, 16), (5, 144, 48), (70, 272, 304), (300, 1040, 128), (777, 512, 1024)])
@pytest.mark.parametrize("act,wd", [(None, F), ("gelu", F), (None, BF)])
def test_training_gradients(m, k, n, act, wd):
    x = workloads.draw("normal_outliers", (m, k), 250, m).to(DEV).requires_grad_()
    w = (workloads.draw("normal", (n, k), 251, n, 0.05).to(DEV).to(wd)).requires_grad_()
    b = workloads.draw("normal", (n,), 252, n).to(DEV).to(wd).requires_grad_()
    res = workloads.draw("normal", (m, n), 253, n).to(DEV).requires_grad_()
    gy = workloads.draw("t3", (m, n), 254, n, 1e-2).to(DEV)
    y = nv().fp8_linear_train(x, w, b, activation=act, residual=res)
    wc, ws, wct, wst = nv().fp8_quantize_weight(w.detach(), transpose=True)
    z = torch.empty(m, n, device=DEV, dtype=BF)
    want = nv().fp8_linear(x.detach(), wc, ws, b.detach().to(BF), activation=act, residual=res.detach(),
                           preact=z if act else None)
    assert torch.equal(y, want)
    gx, gw, gb, gr = torch.autograd.grad(y, (x, w, b, res), gy)
    assert torch.equal(gr, gy) and gx.dtype == BF and gw.dtype == wd and gb.dtype == wd
    g = gy if act is None else nv().activation_backward(gy, nv().checkpoint_pack(z), act)
    gc, gs = nv().fp8_quantize_activation(g)
    gv, wv = _values(gc, gs, False), _values(wc, ws, True)
    _check(gx, gv, np.ascontiguousarray(wv.T))
    xv = _f(nv().checkpoint_pack(x.detach()).dequantized(F)).astype(np.float64)
    g64 = _f(g).astype(np.float64)
    half = 2.0 ** -8 * 1.01 if wd == BF else 2.0 ** -24
    assert np.all(np.abs(_f(gw) - g64.T @ xv) <= (m + 4) * 2.0 ** -23 * (np.abs(g64).T @ np.abs(xv)) + half * np.abs(g64.T @ xv) + 1e-37)
    assert np.all(np.abs(_f(gb) - g64.sum(0)) <= (m + 2) * 2.0 ** -24 * np.abs(g64).sum(0) + half * np.abs(g64.sum(0)))


def test_training_follows_the_full_precision_gradient():
    # quantization taken as the identity: the gradients point where the exact linear's do.  A code is
    # off by 2^-4 of its value at most; independent errors leave a product of random operands within
    # sqrt(2) 2^-4 of itself in norm
    m, k, n = 256, 512, 384
    x, w = torch.randn(m, k, device=DEV).to(BF), torch.randn(n, k, device=DEV) * 0.05
    gy = torch.randn(m, n, device=DEV).to(BF)
    leaves = [x.clone().requires_grad_(), w.clone().requires_grad_()]
    y = nv().fp8_linear_train(*leaves)
    gx, gw = torch.autograd.grad(y, leaves, gy)
    for got, ref in ((y, x.float() @ w.t()), (gx, gy.float() @ w), (gw, gy.float().t() @ x.float())):
        assert (got.float() - ref).norm() <= 2 ** 0.5 * 2.0 ** -4 * ref.norm()


def test_shared_checkpoint_and_partial_gradients():
    m, k, n = 45, 272, 48
    x = torch.randn(m, k, device=DEV).to(BF)
    lw, lb = torch.ones(k, device=DEV, requires_grad=True), torch.zeros(k, device=DEV, requires_grad=True)
    w1, w2 = (torch.randn(n, k, device=DEV).mul_(0.05).requires_grad_() for _ in range(2))
    xl = x.clone().requires_grad_()
    # a pre-norm block: layer norm, two projections on one checkpoint, the second added to the first
    y, ck = nv().layernorm_train(xl, lw, lb, checkpoint=True)
    h = nv().fp8_linear_train(y, w1, checkpoint=ck)
    z = nv().fp8_linear_train(y, w2, checkpoint=ck, activation="silu", residual=h)
    gy = torch.randn_like(z)
    z.backward(gy)
    yd = nv().layernorm(x, lw.detach(), lb.detach())
    ckd = nv().checkpoint_pack(yd)
    assert torch.equal(ckd.codes, ck.codes)
    pre = torch.empty_like(gy)
    nv().fp8_linear(yd, *nv().fp8_quantize_weight(w2.detach()), activation="silu", preact=pre)
    g2 = nv().activation_backward(gy, nv().checkpoint_pack(pre), "silu")
    assert torch.equal(w1.grad, nv().weight_grad(gy, ckd)) and torch.equal(w2.grad, nv().weight_grad(g2, ckd))
    gys = []
    for g, w in ((gy, w1), (g2, w2)):
        _, _, wt, st = nv().fp8_quantize_weight(w.detach(), transpose=True)
        gys.append(nv().fp8_gemm(*nv().fp8_quantize_activation(g), wt, st))
    gx, gw, gb = nv().layernorm_backward((gys[0] + gys[1]), x, lw.detach())
    assert torch.equal(xl.grad, gx) and torch.equal(lw.grad, gw) and torch.equal(lb.grad, gb)
    # gradients of the weight alone, and of the input alone
    w3 = w1.detach().clone().requires_grad_()
    nv().fp8_linear_train(x, w3).backward(gy)
    assert torch.equal(w3.grad, nv().weight_grad(gy, nv().checkpoint_pack(x)))
    x3 = x.clone().requires_grad_()
    nv().fp8_linear_train(x3, w1.detach()).backward(gy)
    assert torch.equal(x3.grad, gys[0])
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(nv().fp8_linear_train(x3, w3).float().square().sum(), x3, create_graph=True)
        g.sum().backward()


def test_training_of_an_empty_batch_and_expanded_gradients():
    w, b = (torch.randn(48, 272, device=DEV) * 0.05).requires_grad_(), torch.zeros(48, device=DEV, requires_grad=True)
    lw, lb = torch.ones(272, device=DEV, requires_grad=True), torch.zeros(272, device=DEV, requires_grad=True)
    x = torch.empty(0, 272, device=DEV, dtype=BF, requires_grad=True)
    y, ck = nv().layernorm_train(x, lw, lb, checkpoint=True)
    nv().fp8_linear_train(y, w, b, checkpoint=ck, activation="gelu").sum().backward()
    assert x.grad.shape == (0, 272)
    for p in (w, b, lw, lb):
        assert p.grad.shape == p.shape and not p.grad.any()
        p.grad = None
    # sum's gradient is one value seen everywhere, through strides of zero
    x = torch.randn(2, 3, 272, device=DEV).to(BF).requires_grad_()
    leaves = (x, w, b, lw, lb)

    def grads(gy):
        y, ck = nv().layernorm_train(x, lw, lb, checkpoint=True)
        return torch.autograd.grad(nv().fp8_linear_train(y, w, b, checkpoint=ck), leaves, gy)

    one = torch.ones(1, device=DEV, dtype=BF).expand(2, 3, 48)
    for got, want in zip(grads(one), grads(one.contiguous())):
        assert torch.equal(got, want)


# ---- streams and graphs ----

@pytest.mark.parametrize("m", [1, 16, 300])
def test_streams_and_graph(m):
    x, (wc, ws), b, res = _case(m, 1040, 528)
    want = nv().fp8_linear(x, wc, ws, b, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = nv().fp8_linear(x, wc, ws, b, residual=res)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv().fp8_linear(x, wc, ws, b, residual=res)
    for i in range(3):
        x.copy_(torch.randn_like(x, dtype=F))
        want = nv().fp8_linear(x, wc, ws, b, residual=res)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_two_captured_graphs_and_training_step_in_a_graph():
    x, (wc, ws), b, res = _case(300, 1040, 528)
    other = _case(300, 1040, 528, 7)[0]
    graphs, ys = [], []
    for t in (x, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(nv().fp8_linear(t, wc, ws, b))
        graphs.append(g)
    want = [nv().fp8_linear(t, wc, ws, b) for t in (x, other)]
    torch.cuda.synchronize()
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(ys, want))
    w = (torch.randn(528, 1040, device=DEV) * 0.05).requires_grad_()
    bias = torch.zeros(528, device=DEV, requires_grad=True)
    xl = x.clone().requires_grad_()
    gy = torch.randn(300, 528, device=DEV).to(BF)

    def step():
        y = nv().fp8_linear_train(xl, w, bias, activation="gelu")
        return (y.detach(), *torch.autograd.grad(y, (xl, w, bias), gy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(3):
        with torch.no_grad():
            xl.copy_(torch.randn(300, 1040, device=DEV))
            gy.copy_(torch.randn(300, 528, device=DEV))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), i
