"""Pins of the oracle's operator definitions: hand values, exhaustive format checks and
gradients against central differences, in float64 on the CPU."""
import numpy as np
import pytest
import torch

import oracle as o


def test_rmsnorm_hand_values():
    # mean square of (3, 4) repeated is 12.5
    r, y = o.rmsnorm(np.array([[3.0, 4.0] * 8]), np.full(16, 2.0), 0.0)
    assert np.array_equal(r, np.array([[3.0, 4.0] * 8], dtype=np.float32))
    s = np.float32(1.0 / np.sqrt(12.5))
    assert np.array_equal(y[0, :2], o.bf16_round(np.array([3.0, 4.0], dtype=np.float32) * s * np.float32(2.0)))
    # eps bounds the scale of a zero row
    assert not o.rmsnorm(np.zeros((1, 16)), np.ones(16), 1e-6)[1].any()


def test_residual_is_rounded_to_the_stream():
    x, res = np.full((1, 16), 2.0 ** -9), np.ones((1, 16))
    assert np.all(o.rmsnorm(x, np.ones(16), 0.0, res, "bf16")[0] == 1.0)
    assert np.all(o.rmsnorm(x, np.ones(16), 0.0, res, "f32")[0] == np.float32(1.0 + 2.0 ** -9))


def test_rmsnorm_grads_against_differences():
    g = np.random.default_rng(3)
    r, w, gy = g.standard_normal((3, 32)), 1 + 0.1 * g.standard_normal(32), g.standard_normal((3, 32))

    def f(r, w):
        return np.sum(gy * r * w / np.sqrt(np.mean(r * r, -1, keepdims=True) + np.float64(np.float32(1e-3))))

    gr, gw = o.rmsnorm_grads(gy, r, w, 1e-3)
    h = 1e-5
    for i in (0, 17, 31):
        d = np.zeros(32)
        d[i] = h
        e = np.zeros((3, 32))
        e[1, i] = h
        assert abs((f(r + e, w) - f(r - e, w)) / (2 * h) - gr[1, i]) < 1e-7
        assert abs((f(r, w + d) - f(r, w - d)) / (2 * h) - gw[i]) < 1e-7


def test_checkpoint_every_code_returns():
    # a block holding +-448 keeps scale 1, and every E4M3 value is its own code
    vals = o.e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64)
    row = np.zeros((1, 32 * 5))
    row[0, :128] = np.concatenate([vals, [0.0]])
    row = row.reshape(5, 32)
    row[:, 31] = 448.0
    codes, scales = o.checkpoint_pack(row.reshape(1, -1))
    assert np.all(scales == 127)
    assert np.array_equal(o.checkpoint_unpack(codes, scales).reshape(5, 32), row)


@pytest.mark.parametrize("top,byte", [(448.0, 127), (448.5, 128), (224.0, 126), (225.0, 127), (1.0, 119), (0.0, 17),
                                      (2.0 ** -130, 17), (1.75 * 2.0 ** 100, 219)])
def test_checkpoint_scale_byte(top, byte):
    x = np.zeros((1, 16))
    x[0, 3] = -top
    assert o.checkpoint_pack(x)[1].tolist() == [[byte]]


def test_checkpoint_rounding_bound_and_torch():
    g = np.random.default_rng(5)
    x = g.standard_normal((64, 80)) * np.exp(4 * g.standard_normal((64, 1)))
    codes, scales = o.checkpoint_pack(x)
    assert scales.shape == (64, 3)
    v = o.checkpoint_unpack(codes, scales)
    s = np.repeat(2.0 ** (scales.astype(float) - 127), 32, 1)[:, :80]
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))
    t = torch.from_numpy(x / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(t, codes)


def test_checkpoint_non_finite():
    x = np.ones((1, 32))
    x[0, 1], x[0, 2], x[0, 3] = np.inf, -np.inf, np.nan
    codes, scales = o.checkpoint_pack(x)
    v = o.checkpoint_unpack(codes, scales)
    assert np.isnan(v[0, 1:4]).all() and np.all(v[0, 4:] == 1.0) and scales[0, 0] == 119


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", None])
def test_activation_grads_against_differences(kind):
    z = np.linspace(-8, 8, 101)
    h = 1e-5
    d = (o.activation(z + h, kind) - o.activation(z - h, kind)) / (2 * h)
    assert np.max(np.abs(d - o.activation_grad(z, kind))) < 1e-9


def test_activations_against_torch():
    z = torch.linspace(-12, 12, 97, dtype=torch.float64)
    f = torch.nn.functional
    for kind, ref in (("silu", f.silu(z)), ("gelu", f.gelu(z)), ("gelu_tanh", f.gelu(z, approximate="tanh"))):
        assert np.allclose(o.activation(z.numpy(), kind), ref.numpy(), rtol=1e-10, atol=1e-13)
