"""The library and the marshalling module are built apart (no GPU)."""
import os
import shutil
import subprocess
import sys

import torch

import speculative_decoding_verification_17_gb300 as sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "speculative_decoding_verification_17_gb300"

PROGRAM = f"""
import {PKG} as sv
assert sv.library().spec_verify_greedy_workspace(4, 3, 1000, 0) > 0  # a call that needs no module
import torch
try:
    sv.logit_adjust(torch.zeros((1, 1, 8)))
except RuntimeError as e:
    assert "binding.cpp" in str(e), e
    print("as it should be")
"""


def test_the_verify_calls_do_not_need_a_host_compiler_for_the_others(tmp_path):
    """A copy of the package with the library built, no module and no compiler for it."""
    sv.library()
    for name in (PKG, "include"):
        shutil.copytree(os.path.join(ROOT, name), tmp_path / name,
                        ignore=shutil.ignore_patterns("_calls*", "__pycache__"))
    so = tmp_path / PKG / "_build" / "libspecverify.so"
    os.utime(so)
    env = {**os.environ, "CXX": "/nonexistent/compiler", "NVCC": "/nonexistent/nvcc"}
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, env=env, capture_output=True,
                       text=True)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stdout + r.stderr
    # with the compiler back the module is built, and named after what it was built against
    r = subprocess.run([sys.executable, "-c", f"import {PKG}._native as n; n.calls(); print(n._calls_path())"],
                       cwd=tmp_path, env={**os.environ, "NVCC": "/nonexistent/nvcc"},
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    path = r.stdout.strip().splitlines()[-1]
    assert torch.__version__ in path and sys.implementation.cache_tag in path and os.path.exists(path)
