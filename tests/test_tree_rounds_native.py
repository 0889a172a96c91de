"""The plan of trees in rounds of whole row tiles (csrc/chunk_plan.h), compiled by
the host compiler: every (row tile, key tile) is covered once, evenly."""
import os
import shutil
import subprocess

import pytest

from _util import ROOT

CSRC = os.path.join(ROOT, "decode_dsa_kv_gb300", "csrc")


def test_rounds_cover_everything_once(tmp_path):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "tree_rounds_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-Wno-unused-function",
                    "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I" + CSRC,
                    os.path.join(ROOT, "tests", "tree_rounds_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), (r.returncode, r.stdout)
