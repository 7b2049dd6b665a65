"""8-bit linears whose caller gives outputs or a workspace that share memory with what the call
reads: the bias, which workgroups read while others write, and the workspace, which holds the
quantized input and partial sums.  On the host, with a library that records launches."""
import os

import pytest
import torch

from nvfp4_w4a4_quantized_global_amd import _lib, fp8
from tests._fake_gpu import install, on_gpu
from tests.test_blocks_host import MODULES

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libnvfp4.so not built")
BF, U8, F = torch.bfloat16, torch.uint8, torch.float32
# one launch without a workspace, streamed rows, tiles split along K
SIZES = [(4, 144, 32), (20, 144, 32), (130, 5120, 256)]


def _z(*shape, dtype=BF):
    return on_gpu(torch.zeros(shape, dtype=dtype))


def _tensors(m, k, n):
    kb, nb = -(-k // 128), -(-n // 128)
    return {"x": _z(m, k), "up": _z(m, k), "codes": _z(n, k, dtype=U8), "scales": _z(nb, kb, dtype=F), "bias": _z(n),
            "residual": _z(m, n), "out": _z(m, n), "preact": _z(m, n), "xc": _z(m, k, dtype=U8), "xs": _z(kb, m, dtype=F),
            "ws": _z(1 << 24, dtype=U8)}


def _call(name, t, **kw):
    kw = {"out": t["out"], "workspace": t["ws"], "residual": t["residual"], "preact": t["preact"], "activation": "silu", **kw}
    w = (t["codes"], t["scales"], t["bias"])
    if name == "fp8_linear":
        return fp8.fp8_linear(t["x"], *w, **kw)
    if name == "fp8_linear_swiglu":
        return fp8.fp8_linear_swiglu(t["x"], t["up"], *w, **kw)
    return fp8.fp8_gemm(t["xc"], t["xs"], *w, **kw)


def _need(name, m, k, n):
    return (fp8.fp8_gemm_workspace_bytes if name == "fp8_gemm" else fp8.fp8_linear_workspace_bytes)(m, k, n)


NAMES = ["fp8_linear", "fp8_linear_swiglu", "fp8_gemm"]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("key", ["out", "preact"])
def test_an_output_over_the_bias(name, key, m, k, n, monkeypatch):
    rec = install(monkeypatch, *MODULES)
    for at in (0, m * n - n, n // 2):                 # the bias at its start, its end, and across it
        t = _tensors(m, k, n)
        room = _z(m * n + n)
        t[key], t["bias"] = on_gpu(room[:m * n].view(m, n)), on_gpu(room[at:at + n])
        with pytest.raises(ValueError, match=f"{key} must not overlap"):
            _call(name, t)
    room = _z(m * n + n)
    t[key], t["bias"] = on_gpu(room[:m * n].view(m, n)), on_gpu(room[m * n:])       # beside each other
    assert not rec.calls
    _call(name, t)
    assert len(rec.calls) == 1


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("name", NAMES)
def test_a_workspace_over_what_the_call_reads_or_writes(name, m, k, n, monkeypatch):
    rec = install(monkeypatch, *MODULES)
    t = _tensors(m, k, n)
    need = _need(name, m, k, n)
    used = {"fp8_linear": ["x"], "fp8_linear_swiglu": ["x", "up"], "fp8_gemm": ["xc", "xs"]}[name]
    for key in used + ["codes", "scales", "bias", "residual", "out", "preact"]:
        size = t[key].numel() * t[key].element_size()
        room = _z(size + need + 4096, dtype=U8)
        inside = on_gpu(room[:size].view(t[key].dtype).view(t[key].shape))
        u = dict(t, **{key: inside})
        after = (size + 255) // 256 * 256
        for at in (0, size - size % 256 - (256 if size % 256 == 0 else 0)):       # its first bytes, and its last
            ws = on_gpu(room[at:at + need + 256])
            if need:
                with pytest.raises(ValueError, match="workspace must not overlap"):
                    _call(name, u, workspace=ws)
                assert not rec.calls, key
            else:                                       # a call that uses none may be given any
                _call(name, u, workspace=ws)
                rec.calls.clear()
        _call(name, u, workspace=on_gpu(room[after:after + need + 256]))
        assert len(rec.calls) == 1, key
        rec.calls.clear()
    # the bytes behind those that the call uses are the caller's: an output there
    room = _z((need + 255) // 256 * 256 + 2 * m * n, dtype=U8)
    out = on_gpu(room[-2 * m * n:].view(BF).view(m, n))
    _call(name, t, workspace=room, out=out)
    assert len(rec.calls) == 1


def test_an_output_over_the_input_alone(monkeypatch):
    """Nothing else is wrong with the call: no residual, no preact, no bias."""
    rec = install(monkeypatch, *MODULES)
    m, k, n = 4, 64, 32
    x = _z(m, k)
    codes, scales = _z(n, k, dtype=U8), _z(1, 1, dtype=F)
    for first in (0, 1, m * k - m * n):
        out = on_gpu(torch.as_strided(x.as_subclass(torch.Tensor), (m, n), (n, 1), first))
        with pytest.raises(ValueError, match="out must not overlap the input"):
            fp8.fp8_linear(x, codes, scales, out=out)
    assert not rec.calls
