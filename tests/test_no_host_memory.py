"""CPU: a refused feed-forward or norm call returns its status also when the host cannot allocate the
error's text (a C caller cannot catch an exception: one that left the library would end its process)."""
import os
import shutil
import subprocess

import pytest

import blockwise_fp8_zero_fold_amd as fz

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")
EINVAL, ESHAPE = -1, -4


def test_refusals_without_host_memory(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "no_host_memory")
    lib = os.path.dirname(fz.lib_path)
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-rdynamic", os.path.join(HERE, "no_host_memory.cpp"), "-L" + lib,
                        "-lfp8z1", f"-Wl,-rpath,{lib}:/opt/rocm/lib", "-Wl,--allow-shlib-undefined", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    lines = [line.split(" ", 2) for line in r.stdout.splitlines()]
    assert len(lines) == 17
    for name, status, text in lines:
        assert int(status) in (EINVAL, ESHAPE) and text, (name, status, text)
