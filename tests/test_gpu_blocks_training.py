"""The training forms of the 8-bit linear and the layer norm: the same values whichever gradients are
asked for, and no work for the others."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


def nv():
    import nvfp4_w4a4_quantized_global_amd as m
    return m


class Launches:
    """The library, with the names and arguments of its calls."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        fn = getattr(self.real, name)
        if name.endswith("_bytes"):
            return fn
        return lambda *args: self.calls.append((name, args)) or fn(*args)

    def names(self):
        names = [n for n, _ in self.calls]
        self.calls.clear()
        return names


@pytest.fixture
def launches(monkeypatch):
    from nvfp4_w4a4_quantized_global_amd import _lib, checkpoint, fp8, layer_norm, norm, nvfp4
    rec = Launches(_lib.lib())
    for m in (nvfp4, norm, checkpoint, fp8, layer_norm):
        monkeypatch.setattr(m, "lib", lambda: rec)
    return rec


def _leaves(m, k, n, wd=F):
    x = workloads.draw("normal_outliers", (m, k), 330, m).to(DEV)
    w = workloads.draw("normal", (n, k), 331, n, 0.05).to(DEV).to(wd)
    b = workloads.draw("normal", (n,), 332, n).to(DEV).to(wd)
    res = workloads.draw("t3", (m, n), 333, n).to(DEV)
    return [t.requires_grad_() for t in (x, w, b, res)]


@pytest.mark.parametrize("m,k,n", [(1, 16, 16), (1, 5120, 1024), (3, 2064, 304), (16, 1040, 48), (40, 1024, 4096), (300, 1040, 528)])
@pytest.mark.parametrize("act", [None, "gelu_tanh"])
def test_an_evaluation_pass(m, k, n, act, launches):
    x, w, b, res = _leaves(m, k, n)
    want = nv().fp8_linear_train(x, w, b, activation=act, residual=res)
    assert want.requires_grad
    held = nv().checkpoint_pack(x.detach())
    launches.calls.clear()
    for guard in (torch.no_grad(), torch.inference_mode()):
        for ck in (None, held):
            with guard:
                y = nv().fp8_linear_train(x, w, b, checkpoint=ck, activation=act, residual=res)
            assert not y.requires_grad and torch.equal(y, want.detach())
            assert launches.names() == ["nvfp4_fp8_quantize_weight", "nvfp4_fp8_linear"]


@pytest.mark.parametrize("act", [None, "silu"])
def test_each_gradient_alone(act, launches):
    m, k, n = 70, 272, 304
    x, w, b, res = _leaves(m, k, n)
    gy = workloads.draw("t3", (m, n), 334, n, 1e-2).to(DEV)
    every = torch.autograd.grad(nv().fp8_linear_train(x, w, b, activation=act, residual=res), (x, w, b, res), gy)
    for i in range(4):
        t = [leaf.detach().clone().requires_grad_(i == j) for j, leaf in enumerate((x, w, b, res))]
        launches.calls.clear()
        y = nv().fp8_linear_train(*t[:3], activation=act, residual=t[3])
        forward = launches.names()
        got, = torch.autograd.grad(y, t[i], gy)
        backward = launches.names()
        assert torch.equal(got, every[i])
        assert ("nvfp4_checkpoint_pack" in forward) == (act is not None and i < 3)
        assert ("nvfp4_fp8_quantize_checkpoint" in forward) == (i == 1)
        want = {0: ["nvfp4_fp8_quantize_activation", "nvfp4_fp8_gemm"], 1: ["nvfp4_weight_grad"],
                2: ["nvfp4_fp8_quantize_activation"], 3: []}[i]
        assert backward == ([] if act is None or i == 3 else ["nvfp4_activation_backward"]) + want


@pytest.mark.parametrize("k", [48, 1040, 5120])
@pytest.mark.parametrize("stream", [None, BF, F])
def test_a_norm_with_frozen_parameters(k, stream):
    m = 37
    x = workloads.draw("normal_outliers", (m, k), 340, m).to(DEV)
    w, b = ((1 + 0.1 * workloads.draw("normal", (k,), 341, i).float()).to(DEV) for i in range(2))
    res = None if stream is None else workloads.draw("t3", (m, k), 342, m).to(DEV).to(stream)
    gy = workloads.draw("normal", (m, k), 343, m).to(DEV)

    def grads(*need):
        t = [leaf.detach().clone().requires_grad_(i in need) for i, leaf in enumerate((x, w, b))]
        out = nv().layernorm_train(*t, 1e-6, res)
        y, extra = (out, ()) if res is None else (out[0], (out[1],))
        return torch.autograd.grad((y, *extra), [t[i] for i in need], (gy, *(torch.ones_like(e) for e in extra)))

    every = grads(0, 1, 2)
    for need in ((0,), (1,), (2,), (0, 1), (0, 2), (1, 2)):
        for i, got in zip(need, grads(*need)):
            assert got.dtype == every[i].dtype and torch.equal(got, every[i])
