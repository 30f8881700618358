"""How the 4-bit cache's write and read kernels find their rows, and the attention
kernel its shares, under AddressSanitizer and UndefinedBehaviorSanitizer (no GPU):
tests/sanitize/store_driver.cpp on sound and on senseless plans."""
import os

import pytest

from tests.test_sanitize_cache_cpu import CLANGXX, ROCM, SAN, _run


@pytest.mark.skipif(not os.path.exists(CLANGXX), reason="ROCm clang++ not found")
def test_store_blocks_and_shares_under_sanitizers(tmp_path):
    obj, exe = str(tmp_path / "store_driver.o"), str(tmp_path / "store_san")
    _run([CLANGXX, "-x", "hip", "--offload-arch=gfx950", f"--rocm-path={ROCM}", "-std=c++17", "-O1", "-g", "-Xclang",
          "-target-feature", "-Xclang", "-packed-fp32-ops", "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address",
          "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all", "-c",
          os.path.join(SAN, "store_driver.cpp"), "-o", obj])
    _run([CLANGXX, "-fsanitize=address,undefined", obj, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe])
    # (leak checking off: the HIP runtime keeps its own allocations to process exit)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    assert "all checks passed" in _run([exe], env=env).stdout
