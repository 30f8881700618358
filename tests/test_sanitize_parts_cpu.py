"""How a batch that shares its first tokens is cut (dequantizing_gemm_amd/csrc/cache_parts.h) under
AddressSanitizer and UndefinedBehaviorSanitizer (no GPU), with tests/sanitize/parts_driver.cpp; and
that the GPU tests' cases have the tile heights that they are there for."""
import os

import pytest

from tests.test_cache_shared_forms_gpu import FORMS, PAYS
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


def plan(driver, case, share_from):
    D, group, affine, heads, ratio, page, _, pages, entries, own, new = case[:11]
    table = max(entries, pages + max(-(-n // page) for n in own))
    return driver(D, group, int(affine), heads, len(own), sum(new), ratio, table, page, share_from)


@pytest.mark.parametrize("case", FORMS, ids=lambda c: f"{c[0]}-{len(c[9])}")
def test_heights_of_the_gpu_cases(driver, case):
    assert plan(driver, case, 1) == [str(case[11]), str(case[12]), "1"]


def test_all_pairs_of_heights_are_there(driver):
    assert {c[11:] for c in FORMS} >= {(128, 128), (16, 128), (32, 128), (128, 32), (128, 16), (32, 16), (16, 32), (32, 32), (16, 16)}


@pytest.mark.parametrize("case", PAYS, ids=lambda c: f"{c[0]}-{len(c[9])}")
def test_cases_that_share_by_themselves(driver, case):
    D, group, affine, heads, ratio, page, _, pages, entries, own, new = case
    got = plan(driver, case, -1)
    assert got != ["apart"] and 100 < int(got[2]) <= pages * page
    assert got[:2] == plan(driver, case, 1)[:2]
