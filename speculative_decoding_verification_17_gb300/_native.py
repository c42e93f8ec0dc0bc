"""Build and load ``libspecverify.so``, the C-ABI library of the verify step, and ``_calls``, the
checks and marshalling of the calls on logits and on the paged cache.

The library is compiled in-tree from ``csrc/`` for sm_103a only (one ``-gencode``), one
nvcc process per translation unit in parallel, and linked against the static CUDA runtime
so loading it needs no CUDA library path. Loading never falls back to anything: a missing
or stale library is an error. ``_calls`` is a Python module against torch's C++ interface, so its
file is named after the versions of both; the calls that do not use it do not need it.
"""
from __future__ import annotations

import ctypes
import glob
import os
import subprocess
import sys
import threading
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
SO = os.path.join(BUILD, "libspecverify.so")
BINDING = os.path.join(CSRC, "binding.cpp")


def _calls_path() -> str:
    import torch

    return os.path.join(BUILD, f"_calls.{sys.implementation.cache_tag}-torch{torch.__version__}.so")


ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "-I", CSRC] + os.environ.get("SV_NVCC_EXTRA", "").split()


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(path: str, deps) -> bool:
    """Whether a built file is missing or older than what it is made of."""
    return not os.path.exists(path) or any(
        os.path.getmtime(d) > os.path.getmtime(path) for d in deps)


def _stale() -> bool:
    return _older(SO, sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _calls_stale() -> bool:
    return _older(_calls_path(), [BINDING] + glob.glob(os.path.join(INCLUDE, "*.h")))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is missing or older than its sources: the library and ``_calls``."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_build_calls) if force or _calls_stale() else None
        if force or _stale():
            _build_library(verbose)
        if binding:
            binding.result()
    return SO


def _build_calls() -> None:
    import sysconfig

    import torch

    os.makedirs(BUILD, exist_ok=True)
    path, root = _calls_path(), os.path.dirname(torch.__file__)
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(root, "include"), "-I",
           os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I",
           sysconfig.get_paths()["include"], BINDING, "-o", tmp, "-L",
           os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{cmd[0]} could not be run on {BINDING}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {BINDING}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def _build_library(verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(16, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = SO + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, SO)


_lock = threading.Lock()
_lib = None
_calls = None


def lib():
    """The loaded library (built first if absent or older than its sources)."""
    global _lib
    with _lock:
        if _lib is None:
            path = SO
            if _stale():
                _build_library(False)
            if not os.path.exists(path):
                raise RuntimeError("libspecverify.so is missing and could not be built")
            L = ctypes.CDLL(path)
            _declare(L)
            _lib = L
    return _lib


def calls():
    """The marshalling module (built first if absent or older than its sources), bound to the loaded
    library."""
    global _calls
    L = lib()
    with _lock:
        if _calls is None:
            import importlib.util

            if _calls_stale():
                _build_calls()
            spec = importlib.util.spec_from_file_location("_calls", _calls_path())
            m = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(m)
            m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                L.logit_adjust, L.paged_attention, L.paged_attention_workspace,
                L.attention_weight_sum, L.kv_cache_evict)))
            _calls = m
    return _calls


class KvPool(ctypes.Structure):
    """sv_kv_pool"""

    _fields_ = [("data", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class KvShape(ctypes.Structure):
    """sv_kv_shape"""

    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "B", "P", "Hq", "Hkv", "D", "page_size",
                                            "num_pages", "max_pages")]


class ScoreRule(ctypes.Structure):
    """sv_score_rule"""

    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int),
                ("slopes", ctypes.c_void_p)]


def _declare(L):
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.sv_version.restype = I
    L.sv_version.argtypes = []
    L.sv_status_string.restype = ctypes.c_char_p
    L.sv_status_string.argtypes = [I]
    L.sv_last_cuda_error.restype = I
    L.sv_last_cuda_error.argtypes = []
    L.spec_verify_sample_workspace.restype = Z
    L.spec_verify_sample_workspace.argtypes = [I, I, I, I]
    L.spec_verify_sample_launches.restype = I
    L.spec_verify_sample_launches.argtypes = [I, I, I, I]
    L.spec_verify_sample.restype = I
    L.spec_verify_sample.argtypes = [P, P, I, P, P, P, I, I, I, F, P, P, P, P, P, P, Z, P]
    L.spec_verify_greedy_workspace.restype = Z
    L.spec_verify_greedy_workspace.argtypes = [I, I, I, I]
    L.spec_verify_greedy.restype = I
    L.spec_verify_greedy.argtypes = [P, I, P, P, I, I, I, P, P, P, Z, P]
    L.spec_verify_greedy_noalloc.restype = I
    L.spec_verify_greedy_noalloc.argtypes = [P, I, P, P, I, I, I, P, P, P]
    L.logit_gap_gate_workspace.restype = Z
    L.logit_gap_gate_workspace.argtypes = [I, I, I]
    L.logit_gap_gate.restype = I
    L.logit_gap_gate.argtypes = [P, I, I, I, F, P, I, P, P, P, P, Z, P]
    L.ngram_propose.restype = I
    L.ngram_propose.argtypes = [P, P, I, I, I, I, I, P, P, P]
    L.draft_confidence_workspace.restype = Z
    L.draft_confidence_workspace.argtypes = [I, I, I, I]
    L.draft_confidence_stop.restype = I
    L.draft_confidence_stop.argtypes = [P, I, P, I, I, I, F, I, F, P, P, P, Z, P]
    D = ctypes.c_double
    L.gate_risk_coverage_workspace.restype = Z
    L.gate_risk_coverage_workspace.argtypes = [I, I]
    L.gate_risk_coverage.restype = I
    L.gate_risk_coverage.argtypes = [P, P, P, I, P, I, P, I, D, D, P, P, P, Z, P]
    L.conformal_residual.restype = I
    L.conformal_residual.argtypes = [P, P, I, I, I, P, P]
    L.conformal_quantile_workspace.restype = Z
    L.conformal_quantile_workspace.argtypes = [I]
    L.conformal_quantile.restype = I
    L.conformal_quantile.argtypes = [P, I, D, P, P, Z, P]
    L.conformal_quantile_barrier_selftest.restype = I
    L.conformal_quantile_barrier_selftest.argtypes = [P, I, P, P, Z, ctypes.c_uint, P]
    L.conformal_admit_workspace.restype = Z
    L.conformal_admit_workspace.argtypes = [I, I, I, I]
    L.conformal_admit.restype = I
    L.conformal_admit.argtypes = [P, I, I, I, I, P, P, P, P, P, Z, P]
    L.ready_cache_record_workspace.restype = Z
    L.ready_cache_record_workspace.argtypes = [I, I, I]
    L.ready_cache_record.restype = I
    L.ready_cache_record.argtypes = [P, P, I, I, P, P, P, P, P, P, I, P, I, I, P, P, P, Z, P]
    L.ready_cache_serve.restype = I
    L.ready_cache_serve.argtypes = [P, P, I, I, P, P, P, P, P, I, F, P, I, I, P, P, P]
    L.ready_cache_invalidate.restype = I
    L.ready_cache_invalidate.argtypes = [P, I, P, P, I, P]
    q = ctypes.c_int64
    L.logit_adjust.restype = I
    L.logit_adjust.argtypes = [P, q, q, I, P, P, P, I, P, P, P, P, P, P, P, I, P, I, I, I, P, q,
                               q, P]
    L.logit_adjust_wait_selftest.restype = I
    L.logit_adjust_wait_selftest.argtypes = [*L.logit_adjust.argtypes[:-1], ctypes.c_uint, P]
    shape = rule = pool = P  # structs: byref() of those above, or their bytes
    L.paged_attention_workspace.restype = Z
    L.paged_attention_workspace.argtypes = [shape]
    L.paged_attention.restype = I
    L.paged_attention.argtypes = [shape, rule, P, q, q, q, pool, pool, P, P, P, P, P, P, Z, P]
    L.attention_weight_sum.restype = I
    L.attention_weight_sum.argtypes = [shape, rule, P, q, q, q, pool, P, P, P, P, q, q, q, P, P,
                                       P, q, P]
    L.paged_attention_wait_selftest.restype = I
    L.paged_attention_wait_selftest.argtypes = [*L.paged_attention.argtypes[:-1], ctypes.c_uint, P]
    L.attention_weight_sum_wait_selftest.restype = I
    L.attention_weight_sum_wait_selftest.argtypes = [*L.attention_weight_sum.argtypes[:-1],
                                                     ctypes.c_uint, P]
    L.kv_cache_evict.restype = I
    L.kv_cache_evict.argtypes = [shape, pool, pool, P, P, P, q, I, I, pool, pool, I, P, I, P, P,
                                 P, P]
