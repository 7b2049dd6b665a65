"""The 8-bit product over the range of its scales: sx * sw is formed in fp32, so blocks whose largest
magnitudes multiply to less than 448^2 2^-126 = 2.3e-33 lose low bits of it, and blocks past
448^2 2^128 = 6.8e43 are outside what the call promises."""
import numpy as np
import pytest
import torch

import workloads
from tests.test_gpu_fp8 import _f, _product, _values, nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
# one launch, streamed with one, two and four tiles of rows, Deep, Small, Large tiles, tiles split along K
SIZES = [(1, 272, 96), (3, 1040, 96), (16, 400, 96), (30, 272, 96), (50, 272, 96), (130, 400, 136), (4400, 272, 520),
         (4352, 272, 4096), (130, 5120, 136)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("xa,wa", [(1e-30, 1.0), (1e-3, 1e-31), (1e-20, 1e-17), (1e-33, 1e-5), (1e-30, 1e-10), (1e12, 1e-36),
                                   (1e20, 1e15), (1e36, 1e-3), (1e-3, 1e36)])
def test_magnitudes(m, k, n, xa, wa):
    """A scale is off by 2^-150 where it is subnormal, against sums of up to 128 448^2: 1.8e-38 a block of
    K.  A subnormal output is off by half its spacing, 2^-134."""
    x = (workloads.draw("normal", (m, k), 350, m).double() * xa).to(BF).to(DEV)
    wc, ws = nv().fp8_quantize_weight((workloads.draw("normal", (n, k), 351, n).double() * wa).float().to(DEV))
    xv, wv = (torch.from_numpy(_values(c, s, w)).to(DEV) for c, s, w in ((*nv().fp8_quantize_activation(x), False), (wc, ws, True)))
    ref, bound = _product(xv, wv)
    got = nv().fp8_linear(x, wc, ws).double()
    blocks = -(-k // 128)
    tol = bound * 1.01 + 2.0 ** -8 * 1.01 * ref.abs() + blocks * 1.8e-38 + 2.0 ** -134
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("m,k,n", SIZES)
def test_sums_of_zero_up_to_the_limit(m, k, n):
    """Blocks whose values multiply to 6e43, each with a sum of exactly 0: 0, and no infinity times it."""
    sign = torch.ones(k)
    sign[1::2] = -1
    for xa, wa in ((1e30, 6e13), (6e13, 1e30), (3e38, 2e5)):
        x = (torch.full((m, k), xa) * sign).to(BF).to(DEV)
        wc, ws = nv().fp8_quantize_weight(torch.full((n, k), wa, device=DEV))
        assert float(x.float().abs().max()) * wa < 6.8e43
        b = workloads.draw("normal", (n,), 352, n).to(DEV)
        assert not nv().fp8_linear(x, wc, ws).any()
        assert torch.equal(nv().fp8_linear(x, wc, ws, b), b.expand(m, n))


def test_small_gradients_train():
    """A training step whose output gradients are 1e-30: those of the input and the weight keep the
    relative error of ordinary ones, since every operand has its own scales."""
    m, k, n = 300, 272, 304
    x, w = torch.randn(m, k, device=DEV).to(BF), torch.randn(n, k, device=DEV) * 0.05
    gy = torch.randn(m, n, device=DEV)
    found = []
    for size in (1.0, 2.0 ** -100):
        t = [x.clone().requires_grad_(), w.clone().requires_grad_()]
        found.append(torch.autograd.grad(nv().fp8_linear_train(*t), t, (gy * size).to(BF)))
    for a, b in zip(*found):
        assert np.array_equal(_f(a), _f(b) * np.float32(2.0 ** 100))
