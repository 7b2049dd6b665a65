"""What the training forms launch: nothing for gradients that nobody can ask for.  On the host, with a
library that records launches."""
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, fp8, layer_norm
from tests._fake_gpu import install, on_gpu
from tests.test_blocks_host import MODULES

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 144, 32
BF = torch.bfloat16
_empty = torch.empty


@pytest.fixture
def rec(monkeypatch):
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: on_gpu(_empty(*s, dtype=dtype)))
    return install(monkeypatch, *MODULES)


def _leaf(*shape, grad=False, dtype=BF):
    return on_gpu(torch.zeros(shape, dtype=dtype)).requires_grad_(grad)


def _names(rec):
    return [name for name, _ in rec.calls]


def _args(rec, name):
    found = [args for n, args in rec.calls if n == name]
    assert len(found) == 1, _names(rec)
    return found[0]


def _step(rec, **need):
    x, w, b, res = (_leaf(*s, grad=need.get(n, False)) for n, s in (("x", (M, K)), ("w", (N, K)), ("b", (N,)), ("res", (M, N))))
    y = fp8.fp8_linear_train(x, w, b, activation="gelu", residual=res)
    return y, (x, w, b, res)


def test_an_evaluation_pass_is_the_inference_linear(rec):
    """Leaves that require gradients, but no graph."""
    for guard in (torch.no_grad(), torch.inference_mode()):
        with guard:
            y, _ = _step(rec, x=True, w=True, b=True, res=True)
        assert y.shape == (M, N) and not y.requires_grad
        assert _names(rec) == ["nvfp4_fp8_quantize_weight", "nvfp4_fp8_linear"]
        assert _args(rec, "nvfp4_fp8_quantize_weight")[-3:-1] == (None, None)          # no transposed codes
        assert _args(rec, "nvfp4_fp8_linear")[10] is None                              # no preact
        rec.calls.clear()


def test_an_evaluation_pass_checks_its_checkpoint(rec):
    from nvfp4_w4a4_quantized_global_amd import checkpoint as ck
    held = ck.Checkpoint(on_gpu(torch.zeros(M + 1, K, dtype=torch.uint8)), on_gpu(torch.zeros(M + 1, 5, dtype=torch.uint8)))
    with torch.no_grad(), pytest.raises(ValueError):
        fp8.fp8_linear_train(_leaf(M, K), _leaf(N, K), checkpoint=held)
    assert not rec.calls


def test_a_gradient_of_the_residual_alone_keeps_no_preactivation(rec):
    y, (_, _, _, res) = _step(rec, res=True)
    assert "nvfp4_checkpoint_pack" not in _names(rec) and _args(rec, "nvfp4_fp8_linear")[10] is None
    rec.calls.clear()
    g = on_gpu(torch.ones(M, N, dtype=BF))
    got, = torch.autograd.grad(y, res, g)
    assert torch.equal(got.as_subclass(torch.Tensor), g.as_subclass(torch.Tensor)) and not rec.calls


@pytest.mark.parametrize("need", ["x", "w", "b"])
def test_a_gradient_behind_the_activation_keeps_it(rec, need):
    _step(rec, **{need: True})
    assert "nvfp4_checkpoint_pack" in _names(rec)
    transposed = _args(rec, "nvfp4_fp8_quantize_weight")[-3]
    assert (transposed is not None) == (need == "x")


@pytest.mark.parametrize("weight,bias", [(False, False), (False, True), (True, False)])
def test_a_frozen_norm_takes_no_parameter_gradients(rec, monkeypatch, weight, bias):
    """A norm whose weight and bias are frozen asks the library for the stream's gradient alone."""
    x, w, b = _leaf(M, K, grad=True), _leaf(K, grad=weight), _leaf(K, grad=bias)
    r = _leaf(M, K)
    ctx = type("Ctx", (), dict(saved_tensors=(r, w), dtypes=(BF, BF, BF), eps=1e-6, has_residual=False,
                               needs_input_grad=(True, weight, bias, False, False, False)))()
    gx, gw, gb, *rest = layer_norm._LayerNormFn.backward(ctx, on_gpu(torch.ones(M, K, dtype=BF)), None, None, None)
    args = _args(rec, "nvfp4_layernorm_backward")
    grads, workspace = args[10:12], args[12:14]
    if weight or bias:
        assert None not in grads and workspace[1] > 0
    else:
        assert grads == (None, None) and workspace == (None, 0)
    assert (gw is None) == (not weight) and (gb is None) == (not bias) and gx.shape == x.shape and rest == [None] * 3
