"""The host code of the norm, epilogue and checkpoint calls under AddressSanitizer and
UndefinedBehaviorSanitizer: tests/test_operators_abi.py against the library that
tests/test_sanitized_abi.py builds (host code only; rebuilt here if it is older than a
source).  Every call returns before a kernel would be queued."""
import glob
import os
import subprocess
import sys

import pytest


def _stale(out, root):
    src = os.path.join(root, "nvfp4_w4a4_quantized_global_amd", "csrc")
    sources = glob.glob(os.path.join(src, "*")) + glob.glob(os.path.join(root, "include", "*.h"))
    return not os.path.exists(out) or any(os.path.getmtime(s) > os.path.getmtime(out) for s in sources)


@pytest.mark.slow
def test_operators_abi_under_host_sanitizers():
    host = pytest.importorskip("tests.test_sanitized_abi")   # a tree for GPU runs may leave it out
    OUT, ROOT = host.OUT, host.ROOT
    runtime = host._asan_runtime()
    if runtime is None:
        pytest.skip("no clang AddressSanitizer runtime under /opt/rocm/llvm")
    if _stale(OUT, ROOT):
        from nvfp4_w4a4_quantized_global_amd import build
        os.makedirs(os.path.dirname(OUT), exist_ok=True)
        build.build(out=OUT, extra_flags=host.HOST_SANITIZE)
    child = (
        "import sys\n"
        f"sys.path.insert(0, {ROOT!r})\n"
        "import nvfp4_w4a4_quantized_global_amd._lib as L\n"
        f"L.LIB_PATH = {OUT!r}\n"
        "import pytest\n"
        "sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', 'tests/test_operators_abi.py']))\n"
    )
    env = dict(os.environ, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:alloc_dealloc_mismatch=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", child], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    report = r.stdout[-4000:] + r.stderr[-4000:]
    assert "ERROR: AddressSanitizer" not in report and "runtime error:" not in report, report
    assert r.returncode == 0 and " passed" in r.stdout, report
