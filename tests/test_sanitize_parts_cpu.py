"""How a batch that shares its first tokens is cut (dequantizing_gemm_amd/csrc/cache_parts.h) under
AddressSanitizer x
import os

import pytest

from tests.test_sanitize_cache_cpu import CLANGXX, ROCM, SAN, _run


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(CLANGXX):
        pytest.skip("ROCm clang++ not found")
    tmp = tmp_path_factory.mktemp("parts")
    obj, exe = str(tmp / "parts.o"), str(tmp / "parts_san")
    _run([CLANGXX, "-x", "hip", "--offload-arch=gfx950", f"--rocm-path={ROCM}", "-std=c++17", "-O1", "-g",
          "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
          "-Xarch_host", "-fno-sanitize-recover=all", "-c", os.path.join(SAN, "parts_driver.cpp"), "-o", obj])
    _run([CLANGXX, "-fsanitize=address,undefined", obj, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib",
          "-lpthread", "-o", exe])
    # (leak checking off: the HIP runtime keeps its own allocations to process exit)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    return lambda *a: _run([exe, *map(str, a)], env=env).stdout.split()


def test_parts_under_sanitizers(driver):
    assert driver() == ["all", "checks", "passed"]

