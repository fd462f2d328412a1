"""The quotients that cut a decode's work (csrc/ranges.h), compiled for the host with checks of signed overflow, with reciprocals
as far off as a kernel's may be (CPU)."""

import os
import shutil
import subprocess

import pytest

from conftest import ROOT


def test_quotients_up_to_int32s_end(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no host compiler")
    exe = tmp_path / "quotient_check"
    cmd = [gxx, "-std=c++17", "-O1", "-fsanitize=undefined,float-cast-overflow", "-fno-sanitize-recover=all", "-static-libubsan",
           f"-I{os.path.join(ROOT, 'paged_kv_cache_126_gb300', 'csrc')}", os.path.join(ROOT, "tests", "c", "quotient_check.cpp"), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout + res.stderr
