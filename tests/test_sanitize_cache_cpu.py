"""The 4-bit cache's host code and the index arithmetic it shares with the kernels
under AddressSanitizer and UndefinedBehaviorSanitizer (no GPU): the entry points
of dequantizing_gemm_amd/csrc/cache_api.cpp with tests/sanitize/cache_driver.cpp,
which stands in for the kernel launchers and checks its own results."""
import os
import subprocess

import pytest

from tests.conftest import ROOT

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CLANGXX = os.path.join(ROCM, "lib", "llvm", "bin", "clang++")
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "dequantizing_gemm_amd", "csrc")


def _run(cmd, env=None):
    r = subprocess.run(cmd, capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, f"{' '.join(cmd)}\nstdout:\n{r.stdout}\nstderr:\n{r.stderr[-4000:]}"
    return r


@pytest.mark.skipif(not os.path.exists(CLANGXX), reason="ROCm clang++ not found")
def test_cache_abi_and_indexing_under_sanitizers(tmp_path):
    hip = [CLANGXX, "-x", "hip", "--offload-arch=gfx950", f"--rocm-path={ROCM}", "-std=c++17", "-O1", "-g",
           "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-c"]
    objs = []
    # api.cpp holds int4_last_error; its own launchers are the stubs of stub_launchers.cpp
    for src in (os.path.join(CSRC, "cache_api.cpp"), os.path.join(CSRC, "api.cpp"),
                os.path.join(SAN, "stub_launchers.cpp"), os.path.join(SAN, "cache_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run(hip + [src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "cache_san")
    _run([CLANGXX, "-fsanitize=address,undefined", *objs, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib",
          "-lpthread", "-o", exe])
    # (leak checking off: the HIP runtime keeps its own allocations to process exit)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    assert "all checks passed" in _run([exe], env=env).stdout
