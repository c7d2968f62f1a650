"""The plans that tests/fp8_plans.py names are those of csrc/fp8_layout.h, and together they reach every
kernel, every tile shape whole and cut along k, and every grouped tile with a loop of its own depth."""

import os
import shutil
import subprocess

import pytest

from fp8_plans import DENSE, GROUPED, RUNS, rows_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("fp8_plans") / "fp8_plan_print")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I" + os.path.join(ROOT, "include"),
           os.path.join(ROOT, "tests", "abi_host", "fp8_plan_print.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(lines):
        got = subprocess.run([out], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [tuple(map(int, ln.split())) for ln in got.stdout.splitlines()]
    return run


def test_dense_plans(ask):
    got = ask([f"dense {m} {n} {k} {int(fast)}" for m, n, k, fast, _ in DENSE])
    assert got == [plan for *_, plan in DENSE]


def test_grouped_tiles(ask):
    lines, want = [], []
    for runs, n, k, exact, fast, bf16 in GROUPED:
        shape = f"grouped {rows_of(runs)} {len(RUNS[runs])} {n}"
        nb = -(-k // 128), -(-2 * k // 128)
        lines += [f"{shape} {nb[0]} 1", f"{shape} {nb[0]} 0", f"{shape} {nb[1]} 0"]
        want += [(exact,), (fast,), (bf16,)]
    assert ask(lines) == want


def test_the_sizes_reach_every_kernel():
    for fast, tiles in ((False, (0, 1, 2, 3)), (True, (0, 1, 2, 3, 4))):
        plans = [p for *_, f, p in DENSE if f == fast]
        for t in tiles:
            assert any(p[0] == 0 and p[1] == t and p[3] for p in plans), (fast, t)      # with parts
        for t in tiles[2:]:
            assert any(p[1] == t and p[2] and not p[3] for p in plans), (fast, t)
            assert any(p[1] == t and p[2] and p[3] for p in plans), (fast, t)           # parts behind whole tiles
    assert any(p[0] for *_, f, p in DENSE if not f)
    # a loop with loads under way through it takes twice the stages in blocks of k
    for column, tiles, blocks in ((3, (0, 1, 3), 128), (4, (0, 1, 2, 4), 128), (5, (0, 1, 2, 4), 64)):
        for t in tiles:
            stages = {0: 3, 1: 3, 2: 4, 3: 3, 4: 2}[t]
            assert any(c[column] == t and -(-c[2] // blocks) >= 2 * stages and c[2] % blocks for c in GROUPED), (column, t)
