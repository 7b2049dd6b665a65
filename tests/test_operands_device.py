"""Operands on another GPU than the call's first tensor are refused before anything is
launched, with or without an epilogue.  On the host, with tensors that say where they are."""
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, checkpoint, nvfp4
from tests._fake_gpu import install, on_gpu

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
M, K, N = 4, 64, 32
BF, U8, F = torch.bfloat16, torch.uint8, torch.float32
SHAPES = {"x": (M, K), "up": (M, K), "codes": (M, K // 2), "packed": (N, K // 2), "bias": (N,), "gx": (), "gw": (),
          "residual": (M, N), "gsf_out": (2,)}


def _calls():
    w = lambda t: (t["packed"], t["inv_scale"], t["gw"], t["bias"], N)  # noqa: E731
    return {
        "linear": (["packed", "inv_scale", "bias", "gx", "gw"],
                   lambda t: nvfp4.nvfp4_linear(t["x"], *w(t), t["gx"], workspace=t["ws"], out=t["out"])),
        "linear_epilogue": (["packed", "inv_scale", "bias", "gx", "gw", "residual"],
                            lambda t: nvfp4.nvfp4_linear(t["x"], *w(t), t["gx"], workspace=t["ws"], out=t["out"],
                                                         residual=t["residual"])),
        "gemm": (["x_scales", "packed", "inv_scale", "bias", "gx", "gw"],
                 lambda t: nvfp4.nvfp4_gemm(t["codes"], t["x_scales"], t["packed"], t["inv_scale"], t["gx"], t["gw"], t["bias"],
                                            out=t["out"], workspace=t["ws"])),
        "swiglu": (["up", "packed", "inv_scale", "bias", "gx", "gw"],
                   lambda t: nvfp4.nvfp4_linear_swiglu(t["x"], t["up"], *w(t), t["gx"], workspace=t["ws"], out=t["out"])),
        "segmented": (["packed", "inv_scale", "bias", "gw", "gsf_out"],
                      lambda t: nvfp4.nvfp4_linear_segmented(t["x"], 2, *w(t), workspace=t["ws"], out=t["out"],
                                                             gsf_out=t["gsf_out"])),
        "noalloc": (["packed", "inv_scale", "bias", "gx", "gw"],
                    lambda t: nvfp4.nvfp4_linear_noalloc(t["x"], *w(t), t["gx"], out=t["out"])),
        "product": (["up"], lambda t: nvfp4.swiglu(t["x"], t["up"])),
        "product and checkpoints": (["up"], lambda t: checkpoint.swiglu_checkpoint(t["x"], t["up"])),
    }


CASES = [(name, other) for name, (operands, _) in _calls().items() for other in [None, *operands]]


@pytest.mark.parametrize("name,elsewhere", CASES)
def test_an_operand_elsewhere_is_refused(name, elsewhere, monkeypatch):
    rec = install(monkeypatch, nvfp4, checkpoint)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: on_gpu(real(*s, dtype=dtype)))
    t = {n: on_gpu(torch.zeros(s, dtype=BF if n in ("x", "up", "bias", "residual") else U8 if n in ("codes", "packed") else F))
         for n, s in SHAPES.items()}
    t["inv_scale"] = on_gpu(torch.zeros(nvfp4.scale_bytes(N, K), dtype=U8))
    t["x_scales"] = on_gpu(torch.zeros(nvfp4.scale_bytes(M, K), dtype=U8))
    t["ws"], t["out"] = on_gpu(torch.zeros(1 << 20, dtype=U8)), on_gpu(torch.zeros((M, N), dtype=BF))
    call = _calls()[name][1]
    if elsewhere is None:
        call(t)
        assert len(rec.calls) == 1
        return
    t[elsewhere] = on_gpu(t[elsewhere], 1)
    with pytest.raises(ValueError, match="cuda:0, got cuda:1"):
        call(t)
    assert not rec.calls
