"""Every call launches with its tensors' device current, however the arguments are given.  On
the host, with tensors that say they are on a second GPU."""
import contextlib
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, checkpoint, norm, nvfp4
from tests._fake_gpu import Recorder, on_gpu

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 64, 32
BF, U8, F = torch.bfloat16, torch.uint8, torch.float32
_empty = torch.empty


def z(*s, dtype=BF):
    return on_gpu(torch.zeros(s, dtype=dtype), 1)


def _calls():
    x, h, g = z(M, K), z(M, K), z(dtype=F)
    nw, gy = z(K), z(M, N)
    w = (z(N, K // 2, dtype=U8), z(nvfp4.scale_bytes(N, K), dtype=U8), g, None, N)
    codes, xs = z(M, K // 2, dtype=U8), z(nvfp4.scale_bytes(M, K), dtype=U8)
    ck = checkpoint.Checkpoint(z(M, K, dtype=U8), z(M, K // 32, dtype=U8))
    z8 = checkpoint.Checkpoint(z(M, N, dtype=U8), z(M, N // 32, dtype=U8))
    return {
        "rmsnorm, eps first": lambda: norm.rmsnorm(eps=1e-5, weight=nw, x=x),
        "quantize_rmsnorm, scale first": lambda: norm.quantize_rmsnorm(global_sf_x=None, x=x, weight=nw),
        "rmsnorm_backward": lambda: norm.rmsnorm_backward(x, h, nw),
        "rmsnorm_train": lambda: norm.rmsnorm_train(x, nw),
        "weight_grad, checkpoint first": lambda: checkpoint.weight_grad(ck=ck, grad_y=gy),
        "activation_backward, activation first": lambda: checkpoint.activation_backward(activation="gelu", z=z8, grad_y=gy),
        "swiglu_backward, checkpoints first": lambda: checkpoint.swiglu_backward(gate=ck, up=ck, grad_x=x),
        "checkpoint_pack, group first": lambda: checkpoint.checkpoint_pack(rotation_group=16, x=x),
        "checkpoint_unpack": lambda: checkpoint.checkpoint_unpack(ck),
        "swiglu_checkpoint": lambda: checkpoint.swiglu_checkpoint(x, h),
        "swiglu_train": lambda: checkpoint.swiglu_train(x, h),
        "swiglu_train, checkpoint": lambda: checkpoint.swiglu_train(x, h, checkpoint=True),
        "swiglu": lambda: nvfp4.swiglu(x, h),
        "quantize_swiglu": lambda: nvfp4.quantize_swiglu(x, h),
        "rotate_activation": lambda: nvfp4.rotate_activation(x, 16),
        "quantize_weight": lambda: nvfp4.quantize_weight(x),
        "quantize_activation": lambda: nvfp4.quantize_activation(x),
        "quantize_activation_segmented": lambda: nvfp4.quantize_activation_segmented(x, 2),
        "dequantize": lambda: nvfp4.dequantize(codes, xs, g),
        "amax": lambda: nvfp4.amax(x),
        "static_global_sf": lambda: nvfp4.static_global_sf(g),
        "scale_to_canonical": lambda: nvfp4.scale_to_canonical(xs, M, K),
        "scale_from_canonical": lambda: nvfp4.scale_from_canonical(z(M, 4, dtype=U8)),
        "nvfp4_gemm": lambda: nvfp4.nvfp4_gemm(codes, xs, w[0], w[1], g, g),
        "nvfp4_linear": lambda: nvfp4.nvfp4_linear(x, *w),
        "nvfp4_linear_swiglu": lambda: nvfp4.nvfp4_linear_swiglu(x, h, *w),
        "nvfp4_linear_segmented": lambda: nvfp4.nvfp4_linear_segmented(x, 2, *w),
        "nvfp4_linear_noalloc": lambda: nvfp4.nvfp4_linear_noalloc(x, *w),
    }


NAMES = [
    "rmsnorm, eps first", "quantize_rmsnorm, scale first", "rmsnorm_backward", "rmsnorm_train", "weight_grad, checkpoint first",
    "activation_backward, activation first", "swiglu_backward, checkpoints first", "checkpoint_pack, group first",
    "checkpoint_unpack", "swiglu_checkpoint", "swiglu_train", "swiglu_train, checkpoint", "swiglu", "quantize_swiglu",
    "rotate_activation", "quantize_weight", "quantize_activation", "quantize_activation_segmented", "dequantize", "amax",
    "static_global_sf", "scale_to_canonical", "scale_from_canonical", "nvfp4_gemm", "nvfp4_linear", "nvfp4_linear_swiglu",
    "nvfp4_linear_segmented", "nvfp4_linear_noalloc",
]


@pytest.mark.parametrize("name", NAMES)
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

    calls = _calls()
    library = Library()
    for m in (nvfp4, norm, checkpoint):
        monkeypatch.setattr(m, "lib", lambda: library)
        monkeypatch.setattr(m, "_stream", lambda device: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: on_gpu(
        _empty(*s, dtype=dtype), torch.device(device).index or 0))
    calls[name]()
    launches = [(n, d) for n, d in seen if not n.endswith("scale_bytes")]
    assert launches and all(d == 1 for _, d in launches), launches
    assert current == [0]
