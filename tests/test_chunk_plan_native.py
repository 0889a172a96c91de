"""The kernel's own plan functions (csrc/chunk_plan.h), compiled by the host
compiler, against counts one by one in 64 bits, up to the largest lengths that
the call takes."""
import os
import shutil
import subprocess

import pytest

from _util import ROOT

CSRC = os.path.join(ROOT, "decode_dsa_kv_gb300", "csrc")


def test_plan_functions_against_counts(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "chunk_plan_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-Wno-unused-function",
                    "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I" + CSRC,
                    os.path.join(ROOT, "tests", "chunk_plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), (r.returncode, r.stdout)
