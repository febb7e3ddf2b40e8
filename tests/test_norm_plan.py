"""CPU: the norm join's launches at every width.  Rows without end give every compute unit the same
number of workgroups, at least one, and no more waves than it holds; few rows give no workgroup
without a row."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")
UNITS, WAVES = 256, 16  # compute units, and waves that one holds of these kernels
WIDTHS = list(range(1, 16385, 37)) + [64, 512, 513, 1024, 4096, 4097, 5120, 6144, 6656, 7168, 7169, 7680, 8192, 8193, 16384]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "norm_plan")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", os.path.join(HERE, "norm_plan.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(sizes):
        out = subprocess.run([exe], input="".join(f"{t} {c}\n" for t, c in sizes), capture_output=True, text=True)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]

    return run


def test_many_rows_fill_every_compute_unit_alike(plan):
    for c, (threads, fwd, rows, bwd) in zip(WIDTHS, plan([(1 << 30, c) for c in WIDTHS])):
        waves = threads // 64
        assert threads % 64 == 0 and threads <= 1024 and threads * (8 if c <= 8192 else 16) >= c, c
        assert fwd % UNITS == 0 and UNITS <= fwd and fwd // UNITS * waves <= WAVES, (c, fwd)
        assert bwd % UNITS == 0 and UNITS <= bwd and bwd // UNITS * waves * rows <= WAVES, (c, rows, bwd)


def test_few_rows(plan):
    sizes = [(t, c) for t in (1, 2, 3, 17, 255, 256, 257, 1000) for c in WIDTHS]
    for (t, c), (threads, fwd, rows, bwd) in zip(sizes, plan(sizes)):
        assert 1 <= fwd <= t and 1 <= bwd and (bwd - 1) * rows < t, (t, c)
        assert rows * threads <= 1024, (t, c)
