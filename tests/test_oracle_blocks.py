"""Pins of the oracle's layer norm and 8-bit block format: hand values, every E4M3 code, and
gradients against central differences, in float64 on the CPU."""
import numpy as np
import torch

import oracle as o


def test_layernorm_hand_values():
    # 1 and 3 alternating: mean 2, variance 1
    r, y = o.layernorm(np.array([[1.0, 3.0] * 8]), np.full(16, 2.0), np.full(16, 0.5), 0.0)
    assert np.array_equal(r, np.array([[1.0, 3.0] * 8], dtype=np.float32))
    assert np.array_equal(y[0], [-1.5, 2.5] * 8)
    # a constant row is its bias, whatever its size
    assert np.all(o.layernorm(np.full((1, 16), 1e20), np.ones(16), np.full(16, 0.25), 1e-6)[1] == 0.25)
    # the residual is rounded to the stream first
    assert np.all(o.layernorm(np.full((1, 16), 2.0 ** -9), np.ones(16), None, 0.5, np.ones((1, 16)))[0] == 1.0)


def test_layernorm_against_torch():
    g = np.random.default_rng(5)
    x, w, b = g.standard_normal((7, 48)).astype(np.float32), g.standard_normal(48), g.standard_normal(48)
    _, y = o.layernorm(x, w.astype(np.float32), b.astype(np.float32), 1e-5)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x).double(), (48,), torch.from_numpy(w), torch.from_numpy(b),
                                         float(np.float32(1e-5))).numpy()
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5)


def test_layernorm_grads_against_differences():
    g = np.random.default_rng(3)
    r, w, b, gy = g.standard_normal((3, 32)), 1 + 0.1 * g.standard_normal(32), g.standard_normal(32), g.standard_normal((3, 32))

    def f(r, w, b):
        c = r - r.mean(-1, keepdims=True)
        return np.sum(gy * (c / np.sqrt((c * c).mean(-1, keepdims=True) + np.float64(np.float32(1e-3))) * w + b))

    gr, gw, gb = o.layernorm_grads(gy, r, w, 1e-3)
    h = 1e-5
    for i in (0, 17, 31):
        d = np.zeros(32)
        d[i] = h
        e = np.zeros((3, 32))
        e[1, i] = h
        assert abs((f(r + e, w, b) - f(r - e, w, b)) / (2 * h) - gr[1, i]) < 1e-7
        assert abs((f(r, w + d, b) - f(r, w - d, b)) / (2 * h) - gw[i]) < 1e-7
        assert abs((f(r, w, b + d) - f(r, w, b - d)) / (2 * h) - gb[i]) < 1e-7
    assert np.array_equal(o.layernorm_grads(gy, r, w, 1e-3, gy)[0], gr + gy)


def test_fp8_blocks():
    grid = o.e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64)
    # every code comes back as itself under a scale of 1/2 (abs-max 224)
    x = np.zeros((1, 256))
    x[0, :127], x[0, 128:255] = grid / 2, -grid / 2
    codes, scales = o.fp8_quantize(x, 1)
    assert np.array_equal(scales, np.full((1, 2), 0.5, dtype=np.float32))
    assert np.array_equal(codes[0, :127], np.arange(127)) and np.array_equal(codes[0, 128:255], np.arange(127) + 128)
    assert np.array_equal(np.abs(o.fp8_values(codes, scales, 1)), np.abs(x))
    # ties to the even code: 17 and 19 lie between 16, 18 and 20
    x = np.array([[448.0, 17.0, 19.0, -17.0]])
    assert np.array_equal(o.fp8_values(*o.fp8_quantize(x, 1), 1)[0], [448.0, 16.0, 20.0, -16.0])
    # zeros and values far below the floor; what is not finite does not enter the scale
    codes, scales = o.fp8_quantize(np.array([[0.0, -0.0, 1e-40]]), 1)
    assert np.array_equal(codes, [[0, 0x80, 0]]) and scales[0, 0] == np.float32(2.0 ** -110)
    codes, scales = o.fp8_quantize(np.array([[np.inf, 448.0, np.nan, -np.inf]]), 1)
    assert np.array_equal(codes, [[0x7F, 0x7E, 0x7F, 0x7F]]) and scales[0, 0] == 1.0
    # a weight's tiles: ragged in both directions
    w = np.ones((130, 144))
    w[:, 128:] = 2.0
    w[128:, :128] = 4.0
    _, scales = o.fp8_quantize(w, 128)
    assert np.array_equal(scales * 448.0, [[1.0, 2.0], [4.0, 2.0]])
    # the error of a code: 2^-4 of the value, or 2^-10 of the scale
    x = np.random.default_rng(1).standard_normal((5, 400)) * np.exp(np.random.default_rng(2).standard_normal((5, 400)) * 4)
    codes, scales = o.fp8_quantize(x, 1)
    s = np.repeat(scales.astype(np.float64), 128, axis=1)[:, :400]
    assert np.all(np.abs(o.fp8_values(codes, scales, 1) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * (1 + 2.0 ** -22))


def test_torch_conversion_agrees():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(9, 272, generator=g).to(torch.bfloat16).float()
    codes, scales = o.fp8_quantize(x.numpy(), 1)
    pad = torch.nn.functional.pad(x, (0, 112)).reshape(9, 3, 128)
    top = pad.abs().amax(-1)
    q = (pad * (torch.tensor(448.0) / top)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(9, -1)[:, :272]
    assert np.array_equal(codes, q.numpy()) and np.array_equal(scales, (top / torch.tensor(448.0)).numpy())
