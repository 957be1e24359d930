"""The order in which the tcgen05 attention kernel issues its products and frees
its K stages, replayed on the host from the header that the kernel uses."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_k_stages_are_freed_after_both_slots(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "wide_order_check")
    build = subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I",
                            os.path.join(ROOT, "permuted_block_sparse_b200", "csrc"),
                            os.path.join(ROOT, "tests", "c_abi", "wide_order_check.cpp"), "-o", exe],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and " 0 failures" in run.stdout, run.stdout + run.stderr
