"""Allocation failures in the block manager's calls on drafted tokens."""
import os
import shutil
import subprocess

import pytest


def test_failed_allocations_leave_no_trace(tmp_path):
    """Every host allocation inside reserve and commit made to fail in turn: an
    error status each time, and the manager as it was."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "bm_tree_alloc_fail")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(root, "include"),
                    os.path.join(root, "tests", "bm_tree_alloc_fail.cpp"),
                    os.path.join(root, "paged_kv_cache_262_gb300", "csrc", "pa_block_manager.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("ok ") and int(r.stdout.split()[1]) >= 5, r.stdout
