"""Host side of the layer norm and 8-bit block calls: operands of another device, outputs and
workspaces that must not be written, and the device that calls launch on.  With tensors that say
where they are and a library that records launches."""
import contextlib
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, checkpoint, fp8, layer_norm, norm, nvfp4
from tests._fake_gpu import Recorder, install, on_gpu

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 144, 32
BF, U8, F = torch.bfloat16, torch.uint8, torch.float32
MODULES = (nvfp4, norm, checkpoint, fp8, layer_norm)
_empty = torch.empty


def _tensors(gpu=0):
    shapes = {"x": (M, K), "up": (M, K), "h": (M, K), "lw": (K,), "lb": (K,), "bias": (N,), "residual": (M, N), "out": (M, N),
              "preact": (M, N), "w": (N, K), "gy": (M, K)}
    t = {n: on_gpu(torch.zeros(s, dtype=BF), gpu) for n, s in shapes.items()}
    t["codes"], t["scales"] = on_gpu(torch.zeros((N, K), dtype=U8), gpu), on_gpu(torch.zeros((1, 2)), gpu)
    t["xc"], t["xs"] = on_gpu(torch.zeros((M, K), dtype=U8), gpu), on_gpu(torch.zeros((2, M)), gpu)
    t["ws"] = on_gpu(torch.zeros(1 << 20, dtype=U8), gpu)
    return t


def _calls():
    e = lambda t: dict(out=t["out"], workspace=t["ws"], activation="silu", residual=t["residual"], preact=t["preact"])  # noqa: E731
    return {
        "fp8_linear": (["codes", "scales", "bias", "residual", "out", "preact", "ws"],
                       lambda t: fp8.fp8_linear(t["x"], t["codes"], t["scales"], t["bias"], **e(t))),
        "fp8_linear_swiglu": (["up", "codes", "scales", "bias", "residual", "out", "preact", "ws"],
                              lambda t: fp8.fp8_linear_swiglu(t["x"], t["up"], t["codes"], t["scales"], t["bias"], **e(t))),
        "fp8_gemm": (["xs", "codes", "scales", "bias", "residual", "out", "preact", "ws"],
                     lambda t: fp8.fp8_gemm(t["xc"], t["xs"], t["codes"], t["scales"], t["bias"], **e(t))),
        "fp8_quantize_swiglu": (["up"], lambda t: fp8.fp8_quantize_swiglu(t["x"], t["up"])),
        "fp8_quantize_checkpoint": ([], lambda t: fp8.fp8_quantize_checkpoint(t["x"])),
        "fp8_dequantize": (["scales"], lambda t: fp8.fp8_dequantize(t["codes"], t["scales"])),
        "layernorm": (["lw", "lb", "h"], lambda t: layer_norm.layernorm(t["x"], t["lw"], t["lb"], 1e-6, t["h"])),
        "layernorm_checkpoint": (["lw", "lb", "h"], lambda t: layer_norm.layernorm_checkpoint(t["x"], t["lw"], t["lb"], 1e-6, t["h"])),
        "quantize_layernorm": (["lw", "lb", "h"], lambda t: layer_norm.quantize_layernorm(t["x"], t["lw"], t["lb"], 1e-6, t["h"])),
        "fp8_quantize_layernorm": (["lw", "lb", "h"],
                                   lambda t: layer_norm.fp8_quantize_layernorm(t["x"], t["lw"], t["lb"], 1e-6, t["h"])),
        "fp8_quantize_rmsnorm": (["lw", "h"], lambda t: layer_norm.fp8_quantize_rmsnorm(t["x"], t["lw"], 1e-6, t["h"])),
        "layernorm_backward": (["x", "lw", "h"], lambda t: layer_norm.layernorm_backward(t["gy"], t["x"], t["lw"], 1e-6, t["h"])),
    }


CASES = [(name, other) for name, (operands, _) in _calls().items() for other in [None, *operands]]


@pytest.mark.parametrize("name,elsewhere", CASES)
def test_an_operand_elsewhere_is_refused(name, elsewhere, monkeypatch):
    rec = install(monkeypatch, *MODULES)
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: on_gpu(_empty(*s, dtype=dtype)))
    t = _tensors()
    call = _calls()[name][1]
    if elsewhere is None:
        call(t)
        assert len(rec.calls) == 1
        return
    t[elsewhere] = on_gpu(t[elsewhere].clone(), 1)
    with pytest.raises(ValueError, match="cuda:[01], got cuda:[01]"):
        call(t)
    assert not rec.calls
    t[elsewhere] = t[elsewhere].as_subclass(torch.Tensor).clone()      # in host memory
    with pytest.raises(ValueError):
        call(t)
    assert not rec.calls


@pytest.mark.parametrize("name", ["fp8_linear", "fp8_linear_swiglu", "fp8_gemm"])
def test_outputs_that_must_not_be_written(name, monkeypatch):
    rec = install(monkeypatch, *MODULES)
    call = _calls()[name][1]
    t = _tensors()
    x = t["xc"] if name == "fp8_gemm" else t["up"] if name == "fp8_linear_swiglu" else t["x"]
    over = lambda s: on_gpu(torch.as_strided(s.view(BF), (M, N), (N, 1), 0))  # noqa: E731
    bad = {"short": on_gpu(torch.zeros((M - 1, N), dtype=BF)), "fp32": on_gpu(torch.zeros((M, N))),
           "strided": on_gpu(torch.zeros((M, 2 * N), dtype=BF)[:, ::2]), "over the input": over(x),
           "over the weight": over(t["codes"]), "over the residual's middle": None}
    base = torch.zeros(2 * M * N, dtype=BF)
    for what, out in bad.items():
        for key in ("out", "preact"):
            u = dict(t)
            if out is None:
                u["residual"], u[key] = on_gpu(base[:M * N].view(M, N)), on_gpu(base[N:N + M * N].view(M, N))
            else:
                u[key] = out
            with pytest.raises(ValueError):
                call(u)
            assert not rec.calls, (what, key)
    # the residual itself is a fine output
    u = dict(t, residual=t["out"])
    assert call(u).data_ptr() == t["out"].data_ptr() and len(rec.calls) == 1
    # a workspace of the wrong kind
    for ws in (on_gpu(torch.zeros(4096, dtype=U8)[::2]), "workspace"):
        with pytest.raises(ValueError):
            call(dict(t, ws=ws))
    assert len(rec.calls) == 1


def test_given_outputs_count_as_changed(monkeypatch):
    install(monkeypatch, *MODULES)
    for name in ("fp8_linear", "fp8_linear_swiglu", "fp8_gemm"):
        t = _tensors()
        before = t["out"]._version, t["preact"]._version
        _calls()[name][1](t)
        assert t["out"]._version > before[0] and t["preact"]._version > before[1]


LAUNCHES = {
    **{name: call for name, (_, call) in _calls().items()},
    "fp8_quantize_activation, sums first": lambda t: fp8.fp8_quantize_activation(column_sum=True, x=t["x"]),
    "fp8_quantize_weight, transposed": lambda t: fp8.fp8_quantize_weight(transpose=True, w=t["w"]),
    "fp8_linear, weight first": lambda t: fp8.fp8_linear(scales=t["scales"], codes=t["codes"], x=t["x"]),
    "FP8Linear": lambda t: fp8.FP8Linear(t["codes"], t["scales"])(t["x"]),
    "FP8Linear.from_weight": lambda t: fp8.FP8Linear.from_weight(t["w"]),
    "layernorm, eps first": lambda t: layer_norm.layernorm(eps=1e-5, weight=t["lw"], x=t["x"]),
    "layernorm_train": lambda t: layer_norm.layernorm_train(t["x"], t["lw"], t["lb"]),
}


@pytest.mark.parametrize("name", list(LAUNCHES))
def test_launches_on_the_tensors_device(name, monkeypatch):
    current, seen = [0], []

    class Library(Recorder):
        def __getattr__(self, attr):
            fn = super().__getattr__(attr)
            return lambda *args: seen.append((attr, current[-1])) or fn(*args)

    @contextlib.contextmanager
    def device(d):
        current.append(torch.device(d).index)
        yield
        current.pop()

    library = Library()
    for m in MODULES:
        monkeypatch.setattr(m, "lib", lambda: library)
        monkeypatch.setattr(m, "_stream", lambda device: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: on_gpu(
        _empty(*s, dtype=dtype), torch.device(device).index or 0))
    LAUNCHES[name](_tensors(1))
    launches = [(n, d) for n, d in seen if not n.endswith("_bytes") or "workspace" in n]
    assert launches and all(d == 1 for _, d in launches), launches
    assert current == [0]


def test_layer_takes_its_codes_types_only():
    scales = torch.ones(1, 2)
    for dt in (torch.uint8, torch.float8_e4m3fn):
        layer = fp8.FP8Linear(torch.zeros(N, K, dtype=U8).view(dt), scales)
        assert layer.codes.dtype == U8 and (layer.out_features, layer.in_features) == (N, K)
    for bad in (torch.zeros(N, K, dtype=U8).view(torch.float8_e4m3fnuz), torch.zeros(N, K, dtype=U8).view(torch.float8_e5m2),
                torch.zeros(N, K, dtype=torch.int8), torch.zeros(N, K // 2, dtype=BF), torch.zeros(N, 20, dtype=U8),
                torch.zeros(N * K, dtype=U8)):
        with pytest.raises(ValueError):
            fp8.FP8Linear(bad, scales)
