"""The argument checks and plans of the e4m3 and grouped products built for the
host alone, under the address and undefined-behaviour sanitizers.

fp8_api.cpp is linked with stand-in launchers and no HIP runtime (the link shows
that no check reaches a HIP function); tests/abi_host/fp8_validation_driver.cpp
runs every entry point over extreme and ordinary counts and holds each accepted
call's plan to what the kernels assume: grids inside their limits, tiles that add
up, parts of at least four blocks, rows of a tile within 32-bit offsets.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gguf_block_quantized_qmv_amd", "csrc")
HOST = os.path.join(ROOT, "tests", "abi_host")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("fp8_host") / "fp8_validation_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror", "-I" + os.path.join(ROOT, "include"),
           os.path.join(CSRC, "fp8_api.cpp"), os.path.join(HOST, "fp8_stub_launchers.cpp"),
           os.path.join(HOST, "fp8_validation_driver.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"host-only build failed (a HIP symbol would fail the link):\n{r.stderr}"
    return out


def test_checks_and_plans_are_sanitizer_clean(driver):
    # verify_asan_link_order=0: the environment may preload libraries of its own ahead of the ASan runtime
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([driver], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("0 failures"), r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr
