"""A serving step's host code over the 4-bit cache, and the index arithmetic that it
shares with the kernels, under AddressSanitizer and UndefinedBehaviorSanitizer (no
GPU): dequantizing_gemm_amd/csrc/cache_step_api.cpp with tests/sanitize/step_driver.cpp,
which stands in for the kernel launchers and checks its own results."""
import os

import pytest

from tests.test_sanitize_cache_cpu import CLANGXX, CSRC, ROCM, SAN, _run


@pytest.mark.skipif(not os.path.exists(CLANGXX), reason="ROCm clang++ not found")
def test_step_under_sanitizers(tmp_path):
    hip = [CLANGXX, "-x", "hip", "--offload-arch=gfx950", f"--rocm-path={ROCM}", "-std=c++17", "-O1", "-g",
           "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-c"]
    objs = []
    # api.cpp holds int4_last_error; its own launchers are the stubs of stub_launchers.cpp
    for src in (os.path.join(CSRC, "cache_step_api.cpp"), os.path.join(CSRC, "api.cpp"),
                os.path.join(SAN, "stub_launchers.cpp"), os.path.join(SAN, "step_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run(hip + [src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "step_san")
    _run([CLANGXX, "-fsanitize=address,undefined", *objs, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib",
          "-lpthread", "-o", exe])
    # (leak checking off: the HIP runtime keeps its own allocations to process exit)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    assert "all checks passed" in _run([exe], env=env).stdout
