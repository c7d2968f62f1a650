"""Types of the e4m3 and grouped products' results, QMM_FAST_SUMS among them: what is refused and the plan of every
accepted call, in a host-only build under the address and undefined-behaviour sanitizers; and pins of the fp64 oracle
by exact rationals."""

import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from oracle import fp8_oracle as o

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gguf_block_quantized_qmv_amd", "csrc")
HOST = os.path.join(ROOT, "tests", "abi_host")


def test_types_and_plans_are_sanitizer_clean(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path / "fp8_types_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror", "-I" + os.path.join(ROOT, "include"),
           os.path.join(CSRC, "fp8_api.cpp"), os.path.join(HOST, "fp8_stub_launchers.cpp"),
           os.path.join(HOST, "fp8_types_driver.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    # verify_asan_link_order=0: the environment may preload libraries of its own ahead of the ASan runtime
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([out], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("0 failures"), r.stdout + r.stderr
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr


def value(code):
    """An e4m3 code as a rational: sign, four exponent bits with bias 7, three mantissa bits."""
    e, m = (code >> 3) & 15, code & 7
    v = Fraction(m, 8) * Fraction(1, 64) if e == 0 else (1 + Fraction(m, 8)) * Fraction(2) ** (e - 7)
    return -v if code & 128 else v


def finite_codes(g, *shape):
    c = g.integers(0, 256, shape, dtype=np.uint8)
    return np.where((c & 127) == 127, c ^ 1, c)


@pytest.mark.parametrize("m,n,k", [(2, 3, 16), (1, 130, 144), (3, 129, 272)])
def test_product_against_rationals(m, n, k):
    g = np.random.default_rng(k)
    x, w = finite_codes(g, m, k), finite_codes(g, n, k)
    xs = g.uniform(0.1, 3, (o.blocks(k), m)).astype(np.float32)
    ws = g.uniform(0.1, 3, (o.blocks(n), o.blocks(k))).astype(np.float32)
    y, mag = o.product(o.rows_f64(x, xs), o.weights_f64(w, ws))
    picks = [(0, 0), (m - 1, n - 1), (0, n // 2), (m // 2, n - 1)]
    for r, i in picks:
        terms = [Fraction(float(xs[b // 128, r])) * Fraction(float(ws[i // 128, b // 128])) * value(int(x[r, b])) * value(int(w[i, b]))
                 for b in range(k)]
        exact, size = sum(terms), sum(abs(t) for t in terms)
        # fp64: a product of four factors and k additions, each within 2^-53
        assert abs(Fraction(float(y[r, i])) - exact) <= (k + 4) * Fraction(1, 2 ** 53) * size
        assert abs(Fraction(float(mag[r, i])) - size) <= (k + 4) * Fraction(1, 2 ** 53) * size


def test_quantiser_against_rationals():
    g = np.random.default_rng(5)
    x = (g.standard_normal((4, 272)) * 10.0 ** g.uniform(-30, 30, (4, 1))).astype(np.float32)
    x[1, :128] = 0
    x[2, 128:256] = np.float32(1e-44) * (np.arange(128) % 3)   # subnormals
    codes, s = o.quant(x)
    for r in range(4):
        for b in range(3):
            part = x[r, b * 128:(b + 1) * 128]
            top = max(abs(Fraction(float(v))) for v in part)
            want = np.float32(float(top / 448)) if top else np.float32(0)
            assert s[b, r] == max(want, np.float32(2.0 ** -126))
            if b == 1 and r == 2 or b == 0 and r == 1:
                assert s[b, r] == np.float32(2.0 ** -126)
            for v, c in zip(part, codes[r, b * 128:(b + 1) * 128]):
                quotient = np.float32(float(Fraction(float(v)) / Fraction(float(s[b, r]))))
                near = [abs(value(i) - Fraction(float(quotient))) for i in range(256) if i & 127 != 127]
                assert abs(value(int(c)) - Fraction(float(quotient))) == min(near)


def test_codes_that_are_not_numbers():
    assert np.isnan(o.decode([0x7F, 0xFF])).all()
    x, w = np.zeros((2, 16), np.uint8), np.full((2, 16), 0x38, np.uint8)
    x[1, 5] = 0x7F
    y, _ = o.product(o.rows_f64(x, np.ones((1, 2))), o.weights_f64(w, np.ones((1, 1))))
    assert (y[0] == 0).all() and np.isnan(y[1]).all()
