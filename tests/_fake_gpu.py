"""Host tests of the binding: tensors in host memory that say they are on a GPU, and a library
that records what would be launched."""
import torch

from nvfp4_w4a4_quantized_global_amd import _lib


class OnGpu(torch.Tensor):
    """A host tensor that reports device cuda:``gpu`` (0)."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", getattr(self, "gpu", 0)))

    def get_device(self):
        return getattr(self, "gpu", 0)


def on_gpu(t, index=0):
    t = t.as_subclass(OnGpu)
    t.gpu = index
    return t


class Recorder:
    """The library with its sizes, and its launches recorded instead of made."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        real = getattr(_lib.lib(), name)
        if name.endswith("_bytes"):
            return real
        return lambda *args: self.calls.append((name, args)) or 0


def install(monkeypatch, *modules, current=0):
    """Recorder in place of the library, for the binding's modules."""
    rec = Recorder()
    for m in modules:
        monkeypatch.setattr(m, "lib", lambda: rec)
        monkeypatch.setattr(m, "_stream", lambda device: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    return rec
