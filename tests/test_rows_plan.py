"""The packed rows' work split (llama_decode_kv_gb300/csrc/rows_plan.h) on the CPU: a C++
harness walks random batches CTA by CTA and checks that every block of every item is visited
exactly once, that partial-state slots never collide and that divided items are found again."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "llama_decode_kv_gb300", "csrc")


def test_rows_plan(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "rows_plan_test")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    os.path.join(HERE, "native", "rows_plan_test.cpp"), "-o", exe], check=True, capture_output=True,
                   text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
