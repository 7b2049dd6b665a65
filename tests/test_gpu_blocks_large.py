"""The layer norm's and the 8-bit blocks' forms on arrays of more than 2^31 values.  No two rows
are alike at a distance of a power of two, so a read from a wrapped offset gives other values, and
memory that an output may come from is filled first, so that a row which is not written shows.
Rows are independent: those at the start, around each wrap and at the end equal a call on them
alone, bit for bit; sums over all rows are compared with float64."""
import pytest
import torch

from tests.test_gpu_fp8 import _check, _product, _values, nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F, U8 = torch.bfloat16, torch.float32, torch.uint8
U = 2.0 ** -24
M, K = 131504, 16384
PERIOD = 509


def _tall(m, k, seed, dtype=BF):
    """A prime number of different rows, repeated under factors and offsets of their own."""
    assert all(2 ** p // k % PERIOD for p in range(28, 34))
    g = torch.Generator(device=DEV).manual_seed(seed)
    block = torch.randn((PERIOD, k), generator=g, device=DEV)
    x = torch.empty((m, k), dtype=dtype, device=DEV)
    for b, i in enumerate(range(0, m, PERIOD)):
        n = min(PERIOD, m - i)
        x[i:i + n] = block[:n] * (1.0 + 0.125 * (b % 11)) + 0.25 * (b % 13)
    return x


def _pick(m, k, last=300):
    """Rows at the start, where offsets in values pass 2^30, 2^31 and 2^32, and at the end."""
    rows = list(range(PERIOD)) + list(range(m - last, m))
    for p in (30, 31, 32):
        rows += range(2 ** p // k - 3, 2 ** p // k + 4)
    return torch.tensor(sorted({r for r in rows if 0 <= r < m}), device=DEV)


def _fill(*sizes):
    """Leaves blocks of these sizes in bytes, filled with 0xFF, to the allocator."""
    torch.cuda.empty_cache()
    held = [torch.full((s,), 0xFF, dtype=U8, device=DEV) for s in sizes]
    torch.cuda.synchronize()
    del held


@pytest.fixture(scope="module")
def tall():
    x = _tall(M, K, 1)
    assert x.numel() > 2 ** 31 + 400 * K
    return x


@pytest.fixture(scope="module")
def params():
    g = torch.Generator(device=DEV).manual_seed(2)
    return 1 + 0.1 * torch.randn(K, generator=g, device=DEV), 0.1 * torch.randn(K, generator=g, device=DEV)


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("stream", [None, BF, F])
def test_norms_forms(tall, params, stream):
    w, b = params
    pick = _pick(M, K)
    res = None if stream is None else _tall(M, K, 3, stream)
    some, some_res = tall[pick], None if res is None else res[pick]
    extra = [] if res is None else [M * K * (2 if stream == BF else 4)]

    _fill(M * K * 2, M * K, *extra)
    got = nv().layernorm_checkpoint(tall, w, b, 1e-6, res)
    want = nv().layernorm_checkpoint(some, w, b, 1e-6, some_res)
    for a, c in zip(got[:-1], want[:-1]):
        assert torch.equal(a[pick], c)
    assert torch.equal(got[-1].codes[pick], want[-1].codes) and torch.equal(got[-1].scales[pick], want[-1].scales)
    del got
    for form, args in ((nv().fp8_quantize_layernorm, (w, b)), (nv().fp8_quantize_rmsnorm, (w,))):
        _fill(M * K, M * K // 32, *extra)
        got, want = form(tall, *args, 1e-6, res), form(some, *args, 1e-6, some_res)
        assert torch.equal(got[0][pick], want[0]) and torch.equal(got[1][:, pick], want[1])
        assert res is None or torch.equal(got[2][pick], want[2])
        del got
    for static in (20.0, None):
        _fill(M * K // 2, M * K // 16, *extra)
        got = nv().quantize_layernorm(tall, w, b, 1e-6, res, static)
        want = nv().quantize_layernorm(some, w, b, 1e-6, some_res, got[2])      # the scale that was used
        assert torch.equal(got[0][pick], want[0])
        assert torch.equal(got[1].view(K // 128, M, 8)[:, pick], want[1].view(K // 128, len(pick), 8))
        assert res is None or torch.equal(got[3][pick], want[3])
        del got


@pytest.mark.parametrize("rd", [BF, F])
def test_norms_gradient(tall, params, rd):
    w, _ = params
    r, pick = _tall(M, K, 4, rd), _pick(M, K)
    for gres in (None, r):
        _fill(M * K * (2 if rd == BF else 4))
        gr, gw, gb = nv().layernorm_backward(tall, r, w, 1e-6, gres)
        assert torch.equal(gr[pick], nv().layernorm_backward(tall[pick], r[pick], w, 1e-6, None if gres is None else gres[pick])[0])
        del gr
    ref_w, ref_b, mag_w, mag_b = (torch.zeros(K, dtype=torch.float64, device=DEV) for _ in range(4))
    for i in range(0, M, 1500):
        rb, gy = r[i:i + 1500].double(), tall[i:i + 1500].double()
        c = rb - rb.mean(1, keepdim=True)
        n = c / torch.sqrt(c.square().mean(1, keepdim=True) + float(torch.tensor(1e-6)))
        t = gy * n
        ref_w, mag_w, ref_b, mag_b = ref_w + t.sum(0), mag_w + t.abs().sum(0), ref_b + gy.sum(0), mag_b + gy.abs().sum(0)
    # three roundings of a term; additions on its way: its workgroup's rows (512 workgroups walk them), then
    # the workgroups' partials in 32 interleaved sets of 16, then the sets
    tol = U * (3 + -(-M // 512) + 16 + 32)
    assert ((gw.double() - ref_w).abs() <= tol * mag_w).all() and ((gb.double() - ref_b).abs() <= tol * mag_b).all()


def test_quantizers(tall):
    pick = _pick(M, K)
    some = tall[pick]
    _fill(M * K, M * K // 32)
    codes, scales, total = nv().fp8_quantize_activation(tall, column_sum=True)
    c, s = nv().fp8_quantize_activation(some)
    assert torch.equal(codes[pick], c) and torch.equal(scales[:, pick], s)
    ref, mag = (torch.zeros(K, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, M, 1500):
        t = tall[i:i + 1500].double()
        ref, mag = ref + t.sum(0), mag + t.abs().sum(0)
    # 64 workgroups walk the rows of each column, eight at a time; then those eight, two of the 64
    # partials, and 32 of their sums
    assert ((total.double() - ref).abs() <= U * (-(-M // 512) + 8 + 2 + 32) * mag).all()
    for dtype in (BF, F):
        _fill(M * K * (2 if dtype == BF else 4))
        v = nv().fp8_dequantize(codes, scales, dtype)
        assert torch.equal(v[pick], nv().fp8_dequantize(c, s, dtype))
        del v
    del codes, scales
    _fill(M * K, M * K // 32)
    got = nv().fp8_quantize_activation(tall)
    assert torch.equal(got[0][pick], c) and torch.equal(got[1][:, pick], s)
    del got
    _fill(M * K, M * K, M * K // 32)
    codes, scales, ck = nv().fp8_quantize_checkpoint(tall)
    want = nv().checkpoint_pack(some)
    assert torch.equal(codes[pick], c) and torch.equal(scales[:, pick], s)
    assert torch.equal(ck.codes[pick], want.codes) and torch.equal(ck.scales[pick], want.scales)
    del codes, scales, ck
    gate = _tall(M, K, 5)
    _fill(M * K, M * K // 32)
    got, want = nv().fp8_quantize_swiglu(gate, tall), nv().fp8_quantize_swiglu(gate[pick], some)
    assert torch.equal(got[0][pick], want[0]) and torch.equal(got[1][:, pick], want[1])


@pytest.mark.parametrize("dtype", [BF, F])
def test_weight(dtype):
    w = _tall(M, K, 6, dtype)
    # whole tiles of 128 rows at the start, around each wrap, and the last, which is short
    parts = [slice(0, 256), slice(2 ** 30 // K - 128, 2 ** 30 // K + 128), slice(2 ** 31 // K - 128, 2 ** 31 // K + 128),
             slice(M // 128 * 128 - 128, M)]
    _fill(M * K, M * K)
    codes, scales, codes_t, scales_t = nv().fp8_quantize_weight(w, transpose=True)
    for p in parts:
        c, s, ct, st = nv().fp8_quantize_weight(w[p], transpose=True)
        tiles = slice(p.start // 128, -(-p.stop // 128))
        assert torch.equal(codes[p], c) and torch.equal(scales[tiles], s)
        assert torch.equal(codes_t[:, p], ct) and torch.equal(scales_t[:, tiles], st)
    del codes_t
    _fill(M * K)
    again, _ = nv().fp8_quantize_weight(w)
    assert torch.equal(again, codes)
    del again
    _fill(M * K * 4)
    v = nv().fp8_dequantize(codes, scales, F)
    for p in parts:
        tiles = slice(p.start // 128, -(-p.stop // 128))
        assert torch.equal(v[p], nv().fp8_dequantize(codes[p], scales[tiles], F))


def _near(got, xc, xs, wc, ws):
    """Within the product's bound (tests/test_gpu_fp8.py) and a rounding to bf16."""
    ref, bound = _product(*(torch.from_numpy(_values(c, s, w)).to(DEV) for c, s, w in ((xc, xs, False), (wc, ws, True))))
    bad = ~((got.double() - ref).abs() <= bound * 1.01 + 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs())
    assert not bad.any(), (int(bad.sum()), torch.argwhere(bad)[:3])


def test_outputs_with_the_epilogue():
    """Outputs, a residual stream updated in place and preactivations past 2^31 values."""
    m, k, n = 70001, 32, 32768
    x = _tall(m, k, 7)
    wc, ws = nv().fp8_quantize_weight(torch.randn(n, k, device=DEV))
    b = torch.randn(n, device=DEV).to(BF)
    res = _tall(m, n, 8)
    rows = sorted({*range(40), *range(2 ** 30 // n - 3, 2 ** 30 // n + 3), *range(2 ** 31 // n - 3, 2 ** 31 // n + 3), *range(m - 40, m)})
    pick = torch.tensor(rows, device=DEV)
    before = res[pick]
    _fill(m * n * 2)
    pre = torch.empty(m, n, device=DEV, dtype=BF)
    y = nv().fp8_linear(x, wc, ws, b, activation="silu", residual=res, out=res, preact=pre)
    assert y.data_ptr() == res.data_ptr()
    xc, xs = nv().fp8_quantize_activation(x[pick])
    _check(y[pick], _values(xc, xs, False), _values(wc, ws, True), b, "silu", before, pre[pick])
    _fill(m * n * 2)
    y = nv().fp8_linear(x, wc, ws)
    _near(y[pick], xc, xs, wc, ws)


@pytest.mark.parametrize("n", [48, 300])
def test_codes_of_the_input(n):
    """The product's own reads of codes past 2^31."""
    m, k = 140000, 16384
    x = _tall(m, k, 9)
    wc, ws = nv().fp8_quantize_weight(torch.randn(n, k, device=DEV) * 0.02)
    pick = _pick(m, k)
    y = nv().fp8_linear(x, wc, ws)
    _near(y[pick], *nv().fp8_quantize_activation(x[pick]), wc, ws)


def test_a_wide_weight():
    """Weight codes past 2^31, for one row, a few and a tile of them."""
    n, k = M, K
    wc, ws = nv().fp8_quantize_weight(_tall(n, k, 10))
    pick = _pick(n, k)
    wv = nv().fp8_dequantize(wc, ws, F)[pick]
    for m in (1, 16, 48, 130):
        x = torch.randn(m, k, device=DEV).to(BF)
        xc, xs = nv().fp8_quantize_activation(x)
        got = nv().fp8_linear(x, wc, ws)[:, pick]
        ref, bound = _product(nv().fp8_dequantize(xc, xs, F).double(), wv.double())
        assert ((got.double() - ref).abs() <= bound * 1.01 + 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs()).all(), m
