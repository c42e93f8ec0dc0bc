"""GB300-native speculative-decoding verify step.

A thin Python binding over ``libspecverify.so`` (C ABI declared in
``include/specverify.h``). Every function here only checks and marshals arguments: the
work runs in the library's sm_103a kernels on the caller's CUDA stream. Tensors are torch
CUDA tensors (PyTorch provides device memory and streams); the binding never computes a
result itself and raises :class:`SVError` on any non-OK status.

Calls (same names as the C ABI):

- :func:`spec_verify_sample` — modified-rejection verify with residual/bonus draw.
- :func:`spec_verify_greedy` — greedy (temperature-0) verify.
- :func:`spec_verify_greedy_noalloc` — the same without a workspace (fixed library scratch).
- :func:`logit_gap_gate`     — top-1/top-2 logit-gap confidence gate.
- :func:`draft_confidence_stop` — variable-length drafting: the first draft position whose
  top probability (or inverse entropy) is below a floor.
- :func:`ngram_propose`      — prompt-lookup n-gram draft proposer.

Gate calibration and the conformal gate (C ABI in ``include/specverify_calib.h``):

- :func:`gate_risk_coverage` — coverage and false-accept risk of the gate over a threshold
  grid, with Wilson intervals, and the smallest threshold within a risk budget.
- :func:`conformal_residual` — sup-norm distance of draft rows from the true rows.
- :func:`conformal_quantile` — the split-conformal quantile of those residuals.
- :func:`conformal_admit`    — the earliest of K layers whose gap clears 2 Q.

Ready-distribution cache (C ABI in ``include/specverify_cache.h``), through
:class:`ReadyCacheTable`, which owns a device-resident table of session slots:

- :meth:`ReadyCacheTable.record`     — pre-position on idle for a batch of sessions.
- :meth:`ReadyCacheTable.serve`      — the confidence-gated fast path for a batch of requests.
- :meth:`ReadyCacheTable.invalidate` — a mutation of the listed sessions' state.

Logits ahead of a verify (C ABI in ``include/specverify_logits.h``):

- :func:`logit_adjust` — repetition, presence and frequency penalties, per-token biases and an
  allowed-token mask over the rows of all k+1 positions.

The paged key-value cache around a verify (C ABI in ``include/specverify_kv.h``):

- :func:`paged_attention`      — attention of the new positions over the cache.
- :func:`attention_weight_sum` — the weight the accepted positions gave each cached key.
- :func:`kv_cache_evict`       — keeps the most recent and the heaviest keys.

The same cache in 8 bits (C ABI in ``include/specverify_kv8.h``):

- :func:`kv_cache_append_q8` — rounds new keys and values to 8 bits, a scale per block and head.
- :func:`paged_attention_q8` — attention of the new positions over it.

What a step does ahead of its attention (C ABI in ``include/specverify_step.h``):

- :func:`kv_page_map`    — pages and slots of the new positions, from the requests' lengths.
- :func:`qk_norm_rotate` — the norm of every query and key head, and its rotation by position.

Workspaces: pass ``workspace=`` (a uint8 CUDA tensor of at least the size the matching
``*_workspace`` query returns, 256-byte aligned, not shared by calls in flight at the same
time; it needs no initialisation), or let the binding keep one cached per (device, stream,
call) that it grows as needed: calls in flight on different streams never share one. A call that
is captured into a CUDA graph gets one of the graph's own memory instead, so replays of different
graphs never share one either, and none is freed under a graph.
"""
from __future__ import annotations

import ctypes
import struct
import threading

import torch

from . import _native

__all__ = [
    "SVError", "SV_F32", "SV_BF16", "SV_MAX_K", "build", "library", "version",
    "spec_verify_sample_workspace", "spec_verify_sample_launches", "spec_verify_sample",
    "spec_verify_greedy_workspace", "spec_verify_greedy", "spec_verify_greedy_noalloc",
    "logit_gap_gate_workspace", "logit_gap_gate", "ngram_propose",
    "SV_CONF_TOP_PROB", "SV_CONF_INV_ENTROPY", "draft_confidence_workspace",
    "draft_confidence_stop", "SV_MAX_TAUS", "CALIB_POINT", "gate_risk_coverage_workspace",
    "gate_risk_coverage", "conformal_residual", "conformal_quantile_workspace",
    "conformal_quantile", "conformal_admit_workspace", "conformal_admit", "gate_points_dict",
    "ReadyCacheTable", "ready_cache_record_workspace", "SV_CACHE_VALID", "SV_CACHE_DECODED",
    "SV_CACHE_CONSUMED", "CACHE_STATS", "SV_F16", "logit_adjust", "paged_attention_workspace",
    "paged_attention", "attention_weight_sum", "kv_cache_evict", "kv_page_map", "qk_norm_rotate",
    "kv_cache_append_q8", "paged_attention_q8_workspace", "paged_attention_q8",
]

SV_F32 = 0
SV_BF16 = 1
SV_F16 = 2
SV_MAX_K = 16
SV_CONF_TOP_PROB = 0
SV_CONF_INV_ENTROPY = 1
SV_MAX_TAUS = 4096
# sv_calib_point as a row of 8 float64-sized fields: the two counts are int64, the six rates
# float64 (view the int64 columns with .view(torch.int64)).
CALIB_POINT = ("accepted", "wrong", "coverage", "cov_lo", "cov_hi", "risk", "risk_lo",
               "risk_hi")

_STATUS = {0: "SV_OK", 1: "SV_ERR_INVALID_ARG", 2: "SV_ERR_UNSUPPORTED", 3: "SV_ERR_WORKSPACE",
           4: "SV_ERR_CUDA", 5: "SV_ERR_TIMEOUT"}


class SVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        L = _native.lib()
        msg = f"{where}: {_STATUS.get(status, status)} ({L.sv_status_string(status).decode()})"
        if status == 4:
            msg += f", cudaError {L.sv_last_cuda_error()}"
        super().__init__(msg)


def build(force: bool = False, verbose: bool = False) -> str:
    return _native.build(force=force, verbose=verbose)


def library():
    return _native.lib()


def version() -> int:
    return library().sv_version()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_cuda(name, t, dtype=None, shape=None, device=None):
    if t is None:
        return
    if (type(t) is torch.Tensor and (dtype is None or t.dtype is dtype)
            and (shape is None or t.shape == shape)
            and (t.device == device if device is not None else t.is_cuda) and t.is_contiguous()
            and t.is_cuda):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream), stream


_ws_lock = threading.Lock()
_ws_cache: dict = {}


def _capturing(handle: int, stream) -> bool:
    """Whether a stream (None: the current one), whose handle is given, is being captured."""
    if stream is None or handle == torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()):
        return torch._C._cuda_isCurrentStreamCapturing()
    with torch.cuda.stream(stream):
        return torch._C._cuda_isCurrentStreamCapturing()


def _workspace(kind: str, nbytes: int, device, stream):
    """Cached zero-filled workspace for (device, stream, kind) of at least ``nbytes`` bytes.
    Calls on one stream run in order, so they may share it; calls on two streams may overlap,
    so each stream has its own."""
    if _capturing(stream.cuda_stream, stream):
        # the graph's memory pool keeps it (one kept here would be shared with whatever else runs on
        # this stream, and freed under the graph once a larger call replaces it)
        with torch.cuda.stream(stream):
            return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    key = (kind, device, stream.cuda_stream)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            with torch.cuda.stream(stream):
                ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            _ws_cache[key] = ws
    return ws


def _ok(status, where):
    if status != 0:
        raise SVError(status, where)


# ------------------------------------------------------------------------------ sampled
def spec_verify_sample_workspace(B: int, k: int, V: int, dtype: int) -> int:
    return int(library().spec_verify_sample_workspace(B, k, V, dtype))


def spec_verify_sample_launches(B: int, k: int, V: int, dtype: int) -> int:
    return int(library().spec_verify_sample_launches(B, k, V, dtype))


def spec_verify_sample(target_logits, draft_logits, draft_tokens, uniforms, temperature: float,
                       num_draft=None, *, out_tokens=None, out_accept_len=None,
                       out_p_draft=None, out_q_draft=None, out_resid_mass=None,
                       want_probs: bool = True, workspace=None, stream=None):
    """Sampled verify. Returns (tokens [B,k+1], accept_len [B], p_draft [B,k] | None,
    q_draft [B,k] | None, resid_mass [B] | None)."""
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = target_logits.device
    code = _dtype_code(target_logits)
    _check_cuda("target_logits", target_logits)
    _check_cuda("draft_logits", draft_logits, target_logits.dtype, (B, k, V), dev)
    _check_cuda("draft_tokens", draft_tokens, torch.int32, (B, k), dev)
    _check_cuda("uniforms", uniforms, torch.float32, (B, k + 1), dev)
    _check_cuda("num_draft", num_draft, torch.int32, (B,), dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_accept_len is None:
        out_accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    if want_probs:
        if out_p_draft is None:
            out_p_draft = torch.empty((B, k), dtype=torch.float32, device=dev)
        if out_q_draft is None:
            out_q_draft = torch.empty((B, k), dtype=torch.float32, device=dev)
        if out_resid_mass is None:
            out_resid_mass = torch.empty((B,), dtype=torch.float32, device=dev)
    _check_cuda("out_tokens", out_tokens, torch.int32, (B, k + 1), dev)
    _check_cuda("out_accept_len", out_accept_len, torch.int32, (B,), dev)
    _check_cuda("out_p_draft", out_p_draft, torch.float32, (B, k), dev)
    _check_cuda("out_q_draft", out_q_draft, torch.float32, (B, k), dev)
    _check_cuda("out_resid_mass", out_resid_mass, torch.float32, (B,), dev)
    h, st = _stream_handle(stream)
    need = spec_verify_sample_workspace(B, k, V, code)
    ws = workspace if workspace is not None else _workspace("sample", need, dev, st)
    _ok(library().spec_verify_sample(
        _ptr(target_logits), _ptr(draft_logits), code, _ptr(draft_tokens), _ptr(num_draft),
        _ptr(uniforms), B, k, V, float(temperature), _ptr(out_tokens), _ptr(out_accept_len),
        _ptr(out_p_draft), _ptr(out_q_draft), _ptr(out_resid_mass), _ptr(ws), ws.numel(), h),
        "spec_verify_sample")
    return out_tokens, out_accept_len, out_p_draft, out_q_draft, out_resid_mass


# ------------------------------------------------------------------------------ greedy
def spec_verify_greedy_workspace(B: int, k: int, V: int, dtype: int) -> int:
    return int(library().spec_verify_greedy_workspace(B, k, V, dtype))


def spec_verify_greedy(target_logits, draft_tokens, num_draft=None, *, out_tokens=None,
                       out_accept_len=None, workspace=None, stream=None):
    """Greedy verify. Returns (tokens [B,k+1], accept_len [B])."""
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = target_logits.device
    code = _dtype_code(target_logits)
    _check_cuda("target_logits", target_logits)
    _check_cuda("draft_tokens", draft_tokens, torch.int32, (B, k), dev)
    _check_cuda("num_draft", num_draft, torch.int32, (B,), dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_accept_len is None:
        out_accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _check_cuda("out_tokens", out_tokens, torch.int32, (B, k + 1), dev)
    _check_cuda("out_accept_len", out_accept_len, torch.int32, (B,), dev)
    h, st = _stream_handle(stream)
    need = spec_verify_greedy_workspace(B, k, V, code)
    ws = workspace if workspace is not None else _workspace("greedy", need, dev, st)
    _ok(library().spec_verify_greedy(
        _ptr(target_logits), code, _ptr(draft_tokens), _ptr(num_draft), B, k, V,
        _ptr(out_tokens), _ptr(out_accept_len), _ptr(ws), ws.numel(), h), "spec_verify_greedy")
    return out_tokens, out_accept_len


def spec_verify_greedy_noalloc(target_logits, draft_tokens, num_draft=None, *, out_tokens=None,
                               out_accept_len=None, stream=None):
    """Greedy verify without a workspace, for callers that cannot allocate device memory:
    it uses the library's fixed 8 MiB scratch array (shapes needing more are rejected).
    Calls that overlap on the GPU share that array and race. Returns (tokens, accept_len)."""
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = target_logits.device
    code = _dtype_code(target_logits)
    _check_cuda("target_logits", target_logits)
    _check_cuda("draft_tokens", draft_tokens, torch.int32, (B, k), dev)
    _check_cuda("num_draft", num_draft, torch.int32, (B,), dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if out_accept_len is None:
        out_accept_len = torch.empty((B,), dtype=torch.int32, device=dev)
    _check_cuda("out_tokens", out_tokens, torch.int32, (B, k + 1), dev)
    _check_cuda("out_accept_len", out_accept_len, torch.int32, (B,), dev)
    h, _ = _stream_handle(stream)
    _ok(library().spec_verify_greedy_noalloc(
        _ptr(target_logits), code, _ptr(draft_tokens), _ptr(num_draft), B, k, V,
        _ptr(out_tokens), _ptr(out_accept_len), h), "spec_verify_greedy_noalloc")
    return out_tokens, out_accept_len


# ------------------------------------------------------------------------------ gate
def logit_gap_gate_workspace(N: int, V: int, dtype: int) -> int:
    return int(library().logit_gap_gate_workspace(N, V, dtype))


def logit_gap_gate(logits, tau: float, answer_set=None, *, out_token=None, out_gap=None,
                   out_fire=None, workspace=None, stream=None):
    """Gate over the rows of ``logits`` [..., V]. Returns (token [N], gap [N], fire [N])."""
    V = logits.shape[-1]
    N = logits.numel() // V if V else 0
    dev = logits.device
    code = _dtype_code(logits)
    _check_cuda("logits", logits)
    if answer_set is not None:
        _check_cuda("answer_set", answer_set, torch.int32, None, dev)
    n_answer = 0 if answer_set is None else answer_set.numel()
    if out_token is None:
        out_token = torch.empty((N,), dtype=torch.int32, device=dev)
    if out_gap is None:
        out_gap = torch.empty((N,), dtype=torch.float32, device=dev)
    if out_fire is None:
        out_fire = torch.empty((N,), dtype=torch.uint8, device=dev)
    _check_cuda("out_token", out_token, torch.int32, (N,), dev)
    _check_cuda("out_gap", out_gap, torch.float32, (N,), dev)
    _check_cuda("out_fire", out_fire, torch.uint8, (N,), dev)
    h, st = _stream_handle(stream)
    need = logit_gap_gate_workspace(N, V, code)
    ws = workspace if workspace is not None else _workspace("gate", need, dev, st)
    _ok(library().logit_gap_gate(
        _ptr(logits), code, N, V, float(tau), _ptr(answer_set), n_answer, _ptr(out_token),
        _ptr(out_gap), _ptr(out_fire), _ptr(ws), ws.numel(), h), "logit_gap_gate")
    return out_token, out_gap, out_fire


# ------------------------------------------------------------------------ gate calibration
def gate_risk_coverage_workspace(N: int, T: int) -> int:
    return int(library().gate_risk_coverage_workspace(N, T))


def gate_risk_coverage(gap, token, full_token, answer_set, taus, z: float = 1.959963984540054,
                       r_max: float = 0.0, *, out_points=None, out_tau_index=None,
                       workspace=None, stream=None):
    """Risk-coverage sweep. Returns (points [T, 8] float64 whose columns are CALIB_POINT, the
    first two holding int64 bits, tau_index [1] int32). ``gate_points_dict`` unpacks them."""
    N = gap.numel()
    T = taus.numel()
    dev = gap.device
    _check_cuda("gap", gap, torch.float32, (N,), dev)
    _check_cuda("token", token, torch.int32, (N,), dev)
    _check_cuda("full_token", full_token, torch.int32, (N,), dev)
    _check_cuda("taus", taus, torch.float32, (T,), dev)
    if answer_set is not None:
        _check_cuda("answer_set", answer_set, torch.int32, None, dev)
    n_answer = 0 if answer_set is None else answer_set.numel()
    if out_points is None:
        out_points = torch.empty((T, 8), dtype=torch.float64, device=dev)
    if out_tau_index is None:
        out_tau_index = torch.empty((1,), dtype=torch.int32, device=dev)
    _check_cuda("out_points", out_points, torch.float64, (T, 8), dev)
    _check_cuda("out_tau_index", out_tau_index, torch.int32, (1,), dev)
    h, st = _stream_handle(stream)
    need = gate_risk_coverage_workspace(N, T)
    ws = workspace if workspace is not None else _workspace("sweep", need, dev, st)
    _ok(library().gate_risk_coverage(
        _ptr(gap), _ptr(token), _ptr(full_token), N, _ptr(answer_set), n_answer, _ptr(taus), T,
        float(z), float(r_max), _ptr(out_points), _ptr(out_tau_index), _ptr(ws), ws.numel(), h),
        "gate_risk_coverage")
    return out_points, out_tau_index


def gate_points_dict(points) -> dict:
    """Columns of gate_risk_coverage's points as CPU tensors (counts as int64)."""
    p = points.detach().cpu()
    out = {}
    for i, name in enumerate(CALIB_POINT):
        col = p[:, i].contiguous()
        out[name] = col.view(torch.int64) if i < 2 else col
    return out


def conformal_residual(draft_logits, true_logits, *, out_resid=None, stream=None):
    """Sup-norm residual of each draft row [..., V] against the true row. Returns [N] fp32."""
    V = draft_logits.shape[-1]
    N = draft_logits.numel() // V if V else 0
    dev = draft_logits.device
    code = _dtype_code(draft_logits)
    _check_cuda("draft_logits", draft_logits)
    _check_cuda("true_logits", true_logits, draft_logits.dtype, tuple(draft_logits.shape), dev)
    if out_resid is None:
        out_resid = torch.empty((N,), dtype=torch.float32, device=dev)
    _check_cuda("out_resid", out_resid, torch.float32, (N,), dev)
    h, _ = _stream_handle(stream)
    _ok(library().conformal_residual(_ptr(draft_logits), _ptr(true_logits), code, N, V,
                                     _ptr(out_resid), h), "conformal_residual")
    return out_resid


def conformal_quantile_workspace(n: int) -> int:
    return int(library().conformal_quantile_workspace(n))


def conformal_quantile(resid, q: float, *, out_q=None, workspace=None, stream=None):
    """Split-conformal quantile of the residuals [n]. Returns Q as a [1] fp32 tensor."""
    n = resid.numel()
    dev = resid.device
    _check_cuda("resid", resid, torch.float32, (n,), dev)
    if out_q is None:
        out_q = torch.empty((1,), dtype=torch.float32, device=dev)
    _check_cuda("out_q", out_q, torch.float32, (1,), dev)
    h, st = _stream_handle(stream)
    need = conformal_quantile_workspace(n)
    ws = workspace if workspace is not None else _workspace("select", need, dev, st)
    _ok(library().conformal_quantile(_ptr(resid), n, float(q), _ptr(out_q), _ptr(ws),
                                     ws.numel(), h), "conformal_quantile")
    return out_q


def conformal_admit_workspace(N: int, K: int, V: int, dtype: int) -> int:
    return int(library().conformal_admit_workspace(N, K, V, dtype))


def conformal_admit(logits, Q, *, out_layer=None, out_token=None, out_gap=None,
                    want_gap: bool = True, workspace=None, stream=None):
    """Conformal gate over logits [N, K, V] and per-layer quantiles Q [K]. Returns (layer [N],
    token [N], gap [N, K] or None)."""
    N, K, V = logits.shape
    dev = logits.device
    code = _dtype_code(logits)
    _check_cuda("logits", logits)
    _check_cuda("Q", Q, torch.float32, (K,), dev)
    if out_layer is None:
        out_layer = torch.empty((N,), dtype=torch.int32, device=dev)
    if out_token is None:
        out_token = torch.empty((N,), dtype=torch.int32, device=dev)
    if out_gap is None and want_gap:
        out_gap = torch.empty((N, K), dtype=torch.float32, device=dev)
    _check_cuda("out_layer", out_layer, torch.int32, (N,), dev)
    _check_cuda("out_token", out_token, torch.int32, (N,), dev)
    _check_cuda("out_gap", out_gap, torch.float32, (N, K), dev)
    h, st = _stream_handle(stream)
    need = conformal_admit_workspace(N, K, V, code)
    ws = workspace if workspace is not None else _workspace("admit", need, dev, st)
    _ok(library().conformal_admit(_ptr(logits), code, N, K, V, _ptr(Q), _ptr(out_layer),
                                  _ptr(out_token), _ptr(out_gap), _ptr(ws), ws.numel(), h),
        "conformal_admit")
    return out_layer, out_token, out_gap


# ---------------------------------------------------------------- ready-distribution cache
SV_CACHE_VALID, SV_CACHE_DECODED, SV_CACHE_CONSUMED = 1, 2, 4
CACHE_STATS = ("pre_positions", "skipped", "consumed", "wasted", "fast", "fall_invalid",
               "fall_ineligible", "fall_gate", "bad")


def ready_cache_record_workspace(M: int, V: int, dtype: int) -> int:
    return int(library().ready_cache_record_workspace(M, V, dtype))


class ReadyCacheTable:
    """A device-resident table of S session slots (32 bytes each), entries of at most
    max_entry tokens, and the table's event counters; with ``keep_dist`` also one stored
    ready row of V logits per session. A new table is empty (zero-filled)."""

    def __init__(self, S: int, max_entry: int, device, *, V: int | None = None,
                 dist_dtype=None, keep_dist: bool = False):
        self.S, self.max_entry = S, max_entry
        self.slots = torch.zeros((S, 4), dtype=torch.int64, device=device)
        self.device = self.slots.device  # with its index ("cuda" -> "cuda:0")
        self.entry_store = torch.zeros((S, max_entry), dtype=torch.int32, device=self.device)
        self.stats = torch.zeros((len(CACHE_STATS),), dtype=torch.int64, device=self.device)
        self.dist = None
        if keep_dist:
            if V is None or dist_dtype is None:
                raise ValueError("keep_dist needs V and dist_dtype")
            self.dist = torch.zeros((S, V), dtype=dist_dtype, device=self.device)

    def record(self, session, end_pos, entry_tokens, entry_len, headroom, ready_logits, *,
               out_status=None, workspace=None, stream=None):
        """Algorithm 1 for M sessions (distinct ids). Returns out_status [M] int32."""
        M, V = ready_logits.shape
        dev = self.device
        code = _dtype_code(ready_logits)
        _check_cuda("ready_logits", ready_logits, None, None, dev)
        _check_cuda("session", session, torch.int32, (M,), dev)
        _check_cuda("end_pos", end_pos, torch.int64, (M,), dev)
        _check_cuda("entry_tokens", entry_tokens, torch.int32, (M, self.max_entry), dev)
        _check_cuda("entry_len", entry_len, torch.int32, (M,), dev)
        _check_cuda("headroom", headroom, torch.int64, (M,), dev)
        if self.dist is not None:
            _check_cuda("dist", self.dist, ready_logits.dtype, (self.S, V), dev)
        if out_status is None:
            out_status = torch.empty((M,), dtype=torch.int32, device=dev)
        _check_cuda("out_status", out_status, torch.int32, (M,), dev)
        h, st = _stream_handle(stream)
        need = ready_cache_record_workspace(M, V, code)
        ws = workspace if workspace is not None else _workspace("record", need, dev, st)
        _ok(library().ready_cache_record(
            _ptr(self.slots), _ptr(self.entry_store), self.S, self.max_entry, _ptr(self.stats),
            _ptr(session), _ptr(end_pos), _ptr(entry_tokens), _ptr(entry_len), _ptr(headroom),
            M, _ptr(ready_logits), code, V, _ptr(self.dist), _ptr(out_status), _ptr(ws),
            ws.numel(), h), "ready_cache_record")
        return out_status

    def serve(self, session, start, req_tokens, req_len, tau: float, answer_set=None, *,
              exact: bool = True, out_token=None, out_reason=None, stream=None):
        """Algorithm 2 for R requests. Returns (token [R], reason [R]) int32."""
        R = session.numel()
        dev = self.device
        _check_cuda("session", session, torch.int32, (R,), dev)
        _check_cuda("start", start, torch.int64, (R,), dev)
        _check_cuda("req_tokens", req_tokens, torch.int32, (R, self.max_entry), dev)
        _check_cuda("req_len", req_len, torch.int32, (R,), dev)
        if answer_set is not None:
            _check_cuda("answer_set", answer_set, torch.int32, None, dev)
        n_answer = 0 if answer_set is None else answer_set.numel()
        if out_token is None:
            out_token = torch.empty((R,), dtype=torch.int32, device=dev)
        if out_reason is None:
            out_reason = torch.empty((R,), dtype=torch.int32, device=dev)
        _check_cuda("out_token", out_token, torch.int32, (R,), dev)
        _check_cuda("out_reason", out_reason, torch.int32, (R,), dev)
        h, _ = _stream_handle(stream)
        _ok(library().ready_cache_serve(
            _ptr(self.slots), _ptr(self.entry_store), self.S, self.max_entry, _ptr(self.stats),
            _ptr(session), _ptr(start), _ptr(req_tokens), _ptr(req_len), R, float(tau),
            _ptr(answer_set), n_answer, 1 if exact else 0, _ptr(out_token), _ptr(out_reason),
            h), "ready_cache_serve")
        return out_token, out_reason

    def invalidate(self, session, *, stream=None):
        """Section 3.6: the listed sessions' state mutated."""
        n = session.numel()
        _check_cuda("session", session, torch.int32, (n,), self.device)
        h, _ = _stream_handle(stream)
        _ok(library().ready_cache_invalidate(_ptr(self.slots), self.S, _ptr(self.stats),
                                             _ptr(session), n, h), "ready_cache_invalidate")

    def state(self) -> dict:
        """The slots' fields as CPU numpy arrays (a device-to-host copy)."""
        import numpy as np

        raw = self.slots.detach().cpu().numpy().tobytes()
        rec = np.frombuffer(raw, dtype=np.dtype([
            ("position", "<i8"), ("gap", "<f8"), ("token", "<i4"), ("entry_len", "<i4"),
            ("flags", "<u4"), ("epoch", "<u4")]))
        return {k: rec[k].copy() for k in rec.dtype.names}

    def counters(self) -> dict:
        vals = self.stats.detach().cpu().tolist()
        return dict(zip(CACHE_STATS, vals))


# ------------------------------------------------------------------------------ confidence
def draft_confidence_workspace(B: int, k: int, V: int, dtype: int) -> int:
    return int(library().draft_confidence_workspace(B, k, V, dtype))


def draft_confidence_stop(draft_logits, temperature: float, mode: int, floor: float,
                          num_draft=None, *, out_num_draft=None, out_conf=None,
                          want_conf: bool = True, workspace=None, stream=None):
    """Variable-length drafting over draft logits [B, k, V]. Returns (num_draft [B] int32,
    conf [B, k] fp32 or None)."""
    B, k, V = draft_logits.shape
    dev = draft_logits.device
    code = _dtype_code(draft_logits)
    _check_cuda("draft_logits", draft_logits)
    _check_cuda("num_draft", num_draft, torch.int32, (B,), dev)
    if out_num_draft is None:
        out_num_draft = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_conf is None and want_conf:
        out_conf = torch.empty((B, k), dtype=torch.float32, device=dev)
    _check_cuda("out_num_draft", out_num_draft, torch.int32, (B,), dev)
    _check_cuda("out_conf", out_conf, torch.float32, (B, k), dev)
    h, st = _stream_handle(stream)
    need = draft_confidence_workspace(B, k, V, code)
    ws = workspace if workspace is not None else _workspace("conf", need, dev, st)
    _ok(library().draft_confidence_stop(
        _ptr(draft_logits), code, _ptr(num_draft), B, k, V, float(temperature), int(mode),
        float(floor), _ptr(out_num_draft), _ptr(out_conf), _ptr(ws), ws.numel(), h),
        "draft_confidence_stop")
    return out_num_draft, out_conf


# ------------------------------------------------------------------------------ n-gram
def ngram_propose(history, hist_len, n_max: int, n_min: int, k: int, *, out_draft=None,
                  out_num_draft=None, stream=None):
    """Prompt-lookup proposer. Returns (draft [B,k] int32, num_draft [B] int32)."""
    B, L_max = history.shape
    dev = history.device
    _check_cuda("history", history, torch.int32)
    _check_cuda("hist_len", hist_len, torch.int32, (B,), dev)
    if out_draft is None:
        out_draft = torch.empty((B, k), dtype=torch.int32, device=dev)
    if out_num_draft is None:
        out_num_draft = torch.empty((B,), dtype=torch.int32, device=dev)
    _check_cuda("out_draft", out_draft, torch.int32, (B, k), dev)
    _check_cuda("out_num_draft", out_num_draft, torch.int32, (B,), dev)
    h, _ = _stream_handle(stream)
    _ok(library().ngram_propose(_ptr(history), _ptr(hist_len), B, L_max, n_max, n_min, k,
                                _ptr(out_draft), _ptr(out_num_draft), h), "ngram_propose")
    return out_draft, out_num_draft


def _made(make, shape, dtype, device, stream):
    """A new tensor (torch.empty or torch.zeros) of the stream the call runs on: what fills it runs
    there, and the allocator hands out no block that another stream still uses."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


# ------------------------------------------------------------------------------ logits
def logit_adjust(logits, history=None, hist_len=None, *, prompt_len=None, draft_tokens=None,
                 num_draft=None, repetition=None, presence=None, frequency=None,
                 bias_tokens=None, bias_values=None, allowed=None, out=None, stream=None):
    """Penalties, biases and the allowed-token mask over logits [B, P, V], whose rows may lie
    apart (last dimension contiguous). ``allowed`` holds bits, [B, P, ceil(V/32)] int32.
    Returns the adjusted logits [B, P, V] (``out``, which may be ``logits`` itself; rows past a
    request's num_draft are left as they are in it)."""
    if out is None and isinstance(logits, torch.Tensor):
        out = _made(torch.empty, logits.shape, logits.dtype, logits.device, stream)
    status = (_native._calls or _native.calls()).adjust(
        logits, history, hist_len, prompt_len, draft_tokens, num_draft, repetition, presence,
        frequency, bias_tokens, bias_values, allowed, out, _raw_stream(stream, logits))
    if status is not None:
        if status:
            raise SVError(status, "logit_adjust")
        return out
    # an argument that does not fit: the checks one by one
    B, P, V = logits.shape
    dev = logits.device
    code = _dtype_code(logits)
    _check_strided("logits", logits)
    L_max = 0
    if history is not None:
        L_max = history.shape[-1]
        _check_cuda("history", history, torch.int32, (B, L_max), dev)
    _check_cuda("hist_len", hist_len, torch.int32, (B,), dev)
    _check_cuda("prompt_len", prompt_len, torch.int32, (B,), dev)
    _check_cuda("draft_tokens", draft_tokens, torch.int32, (B, P - 1), dev)
    _check_cuda("num_draft", num_draft, torch.int32, (B,), dev)
    _check_cuda("repetition", repetition, torch.float32, (B,), dev)
    _check_cuda("presence", presence, torch.float32, (B,), dev)
    _check_cuda("frequency", frequency, torch.float32, (B,), dev)
    n_bias = 0
    if bias_tokens is not None:
        n_bias = bias_tokens.shape[-1]
        _check_cuda("bias_tokens", bias_tokens, torch.int32, (B, n_bias), dev)
    _check_cuda("bias_values", bias_values, torch.float32, (B, n_bias), dev)
    if n_bias == 0:
        bias_tokens = bias_values = None
    _check_cuda("allowed", allowed, torch.int32, (B, P, (V + 31) // 32), dev)
    _check_strided("out", out, logits.dtype, (B, P, V), dev)
    a, b, _ = logits.stride()
    c, d, _ = out.stride()
    _ok(library().logit_adjust(
        logits.data_ptr(), a, b, code, _ptr(history), _ptr(hist_len),
        _ptr(prompt_len), L_max, _ptr(draft_tokens), _ptr(num_draft), _ptr(repetition),
        _ptr(presence), _ptr(frequency), _ptr(bias_tokens), _ptr(bias_values), n_bias,
        _ptr(allowed), B, P, V, out.data_ptr(), c, d, _raw_stream(stream, logits)),
        "logit_adjust")
    return out


# ------------------------------------------------------------------------------ paged cache
def _check_strided(name, t, dtype=None, shape=None, device=None, last=True):
    """As _check_cuda, for a tensor of which at most the last dimension must be contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if last and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _raw_stream(stream, like):
    """The handle of a stream; for None, of the current one of a tensor's device."""
    if stream is not None:
        return stream.cuda_stream
    if not like.is_cuda:
        return 0  # (refused by the checks)
    return torch._C._cuda_getCurrentRawStream(like.get_device())


# the C structs of specverify_kv.h as bytes
_pack_pool = struct.Struct("@Pqqq").pack
_pack_shape = struct.Struct("@9i").pack
_pack_rule = struct.Struct("@ffiP").pack
_KV_DTYPE = {torch.bfloat16: SV_BF16, torch.float16: SV_F16}


def _kv_pool(name, t, like):
    """A pool [pages, page_size, Hkv, D] of k_cache's type, device and last three sizes."""
    _check_strided(name, t, like.dtype, None, like.device)
    if t.ndim != 4 or t.shape[1:] != like.shape[1:]:
        raise ValueError(f"{name} must have shape [pages, {tuple(like.shape[1:])}], "
                         f"got {tuple(t.shape)}")
    a, b, c, _ = t.stride()
    return _pack_pool(t.data_ptr(), a, b, c)


def _kv_call(q, k_cache, page_table, seq_len, num_draft, slopes, scale, softcap, window):
    """Checks what the calls with queries share; returns their first arguments and sizes."""
    B, P, Hq, D = q.shape
    pages, page_size, Hkv, d = k_cache.shape
    dev = q.device
    dtype = _KV_DTYPE.get(q.dtype)
    if dtype is None:
        raise TypeError(f"queries must be bfloat16 or float16, got {q.dtype}")
    _check_strided("q", q)
    if d != D or k_cache.dtype is not q.dtype or k_cache.device != dev:
        raise ValueError("k_cache must have q's width, type and device")
    _check_cuda("page_table", page_table, torch.int32, (B, page_table.shape[-1]), dev)
    _check_cuda("seq_len", seq_len, torch.int32, (B,), dev)
    _check_cuda("num_draft", num_draft, torch.int32, (B,), dev)
    _check_cuda("slopes", slopes, torch.float32, (Hq,), dev)
    shape = _pack_shape(dtype, B, P, Hq, Hkv, D, page_size, pages, page_table.shape[1])
    rule = _pack_rule(D ** -0.5 if scale is None else scale, softcap, window,
                      0 if slopes is None else slopes.data_ptr())
    a, b, c, _ = q.stride()
    head = (shape, rule, q.data_ptr(), a, b, c, _kv_pool("k_cache", k_cache, k_cache))
    return head, B, P, Hq, Hkv, D, dev


def paged_attention_workspace(B: int, P: int, Hq: int, k_cache, page_table) -> int:
    pages, page_size, Hkv, D = k_cache.shape
    return int(library().paged_attention_workspace(
        _pack_shape(_KV_DTYPE[k_cache.dtype], B, P, Hq, Hkv, D, page_size, pages,
                    page_table.shape[1])))


def paged_attention(q, k_cache, v_cache, page_table, seq_len, *, num_draft=None, scale=None,
                    softcap: float = 0.0, window: int = 0, slopes=None, out=None, out_lse=None,
                    want_lse: bool = True, workspace=None, stream=None):
    """Attention of q [B, P, Hq, D] over a paged cache: k_cache and v_cache are views [pages,
    page_size, Hkv, D] of any page, token and head stride, page_table [B, max_pages] int32,
    seq_len [B] int32 (the new positions included). ``scale`` defaults to D ** -0.5. Returns
    (out [B, P, Hq, D], lse [B, P, Hq] fp32 or None)."""
    if out is None:
        out = _made(torch.empty, q.shape, q.dtype, q.device, stream)
    if out_lse is None and want_lse:
        out_lse = _made(torch.empty, q.shape[:3], torch.float32, q.device, stream)
    h = _raw_stream(stream, q)
    ws = workspace
    if ws is None:
        ws = _ws_cache.get(("attention", q.get_device(), h))
        if ws is not None and _capturing(h, stream):
            ws = None
    fast = (_native._calls or _native.calls()).attention
    status = fast(q, k_cache, page_table, seq_len, num_draft, slopes, scale, softcap, window,
                  v_cache, out, out_lse, ws, h)
    if status is not None and status < 0 and workspace is None:
        # a first call on this stream, one that needs more than the earlier ones did, or a captured one
        ws = _workspace("attention", -status - 1, q.device,
                        stream or torch.cuda.current_stream(q.device))
        if _ws_cache.get(("attention", q.device, h)) is ws:
            _ws_cache["attention", q.get_device(), h] = ws
        status = fast(q, k_cache, page_table, seq_len, num_draft, slopes, scale, softcap, window,
                      v_cache, out, out_lse, ws, h)
    if status is not None:
        if status:
            raise SVError(status if status > 0 else 3, "paged_attention")
        return out, out_lse
    # an argument that does not fit: the checks one by one
    head, B, P, Hq, _, D, dev = _kv_call(q, k_cache, page_table, seq_len, num_draft, slopes,
                                         scale, softcap, window)
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must have k_cache's shape")
    _check_cuda("out", out, q.dtype, (B, P, Hq, D), dev)
    _check_cuda("out_lse", out_lse, torch.float32, (B, P, Hq), dev)
    _check_cuda("workspace", workspace, None, None, dev)
    L = library()
    if workspace is None:
        ws = _workspace("attention", L.paged_attention_workspace(head[0]), dev,
                        stream or torch.cuda.current_stream(dev))
    _ok(L.paged_attention(
        *head, _kv_pool("v_cache", v_cache, k_cache), page_table.data_ptr(), seq_len.data_ptr(),
        _ptr(num_draft), out.data_ptr(), _ptr(out_lse), ws.data_ptr(),
        ws.numel() * ws.element_size(), h), "paged_attention")
    return out, out_lse


def attention_weight_sum(q, k_cache, page_table, seq_len, lse, *, num_draft=None,
                         accept_len=None, scale=None, softcap: float = 0.0, window: int = 0,
                         slopes=None, prior=None, out=None, stream=None):
    """Adds to ``prior`` [B, Hkv, N] fp32 (zeros if None) the softmax weight that the rows up to
    accept_len gave each cached key, with ``lse`` [B, P, Hq] as paged_attention returned it.
    Returns the sums [B, Hkv, N] (``out``, which may be ``prior``)."""
    if out is None:
        N = page_table.shape[-1] * k_cache.shape[1] if prior is None else prior.shape[-1]
        out = _made(torch.zeros, (q.shape[0], k_cache.shape[2], N), torch.float32, q.device, stream)
    h = _raw_stream(stream, q)
    status = (_native._calls or _native.calls()).weights(
        q, k_cache, page_table, seq_len, num_draft, slopes, scale, softcap, window, lse,
        accept_len, prior, out, h)
    if status is not None:
        if status:
            raise SVError(status, "attention_weight_sum")
        return out
    # an argument that does not fit: the checks one by one
    head, B, P, Hq, Hkv, D, dev = _kv_call(q, k_cache, page_table, seq_len, num_draft, slopes,
                                           scale, softcap, window)
    N = out.shape[-1]
    _check_strided("lse", lse, torch.float32, (B, P, Hq), dev, last=False)
    _check_cuda("accept_len", accept_len, torch.int32, (B,), dev)
    _check_cuda("prior", prior, torch.float32, (B, Hkv, N), dev)
    _check_cuda("out", out, torch.float32, (B, Hkv, N), dev)
    _ok(library().attention_weight_sum(
        *head, page_table.data_ptr(), seq_len.data_ptr(), _ptr(num_draft), lse.data_ptr(),
        *lse.stride(), _ptr(accept_len), _ptr(prior), out.data_ptr(), N, h),
        "attention_weight_sum")
    return out


def kv_cache_evict(k_cache, v_cache, page_table, seq_len, weights, budget: int, recent: int,
                   new_k, new_v, new_page_table, *, out_len=None, out_index=None,
                   out_weights=None, stream=None):
    """Keeps min(seq_len, budget) keys of every request and kv head, the last ``recent`` and the
    heaviest others by ``weights`` [B, Hkv, N] fp32, and copies them in order to the pages of
    new_page_table in new_k and new_v (which may be the same pools). Returns (out_len [B],
    out_index [B, Hkv, budget] int32, out_weights [B, Hkv, budget] fp32)."""
    if stream is not None and (out_len is None or out_index is None or out_weights is None):
        with torch.cuda.stream(stream):  # (what is made here belongs to the call's stream)
            return kv_cache_evict(k_cache, v_cache, page_table, seq_len, weights, budget, recent,
                                  new_k, new_v, new_page_table, out_len=out_len,
                                  out_index=out_index, out_weights=out_weights)
    h = _raw_stream(stream, k_cache)
    made = (_native._calls or _native.calls()).evict(
        k_cache, v_cache, page_table, seq_len, weights, budget, recent, new_k, new_v,
        new_page_table, out_len, out_index, out_weights, h)
    if made is not None:
        if made[0]:
            raise SVError(made[0], "kv_cache_evict")
        return made[1:]
    # an argument that does not fit: the checks one by one
    B, max_pages = page_table.shape
    pages, page_size, Hkv, D = k_cache.shape
    dev = k_cache.device
    N = weights.shape[-1]
    new_cols = new_page_table.shape[-1]
    dtype = _KV_DTYPE.get(k_cache.dtype)
    if dtype is None:
        raise TypeError(f"keys and values must be bfloat16 or float16, got {k_cache.dtype}")
    pools = [_kv_pool(name, t, k_cache) for name, t in
             (("k_cache", k_cache), ("v_cache", v_cache), ("new_k", new_k), ("new_v", new_v))]
    if v_cache.shape[0] != pages or new_v.shape[0] != new_k.shape[0]:
        raise ValueError("keys and values must have the same number of pages")
    _check_cuda("page_table", page_table, torch.int32, (B, max_pages), dev)
    _check_cuda("seq_len", seq_len, torch.int32, (B,), dev)
    _check_cuda("weights", weights, torch.float32, (B, Hkv, N), dev)
    _check_cuda("new_page_table", new_page_table, torch.int32, (B, new_cols), dev)
    if not 1 <= budget <= new_cols * page_size:
        raise SVError(1, "kv_cache_evict")
    if out_len is None:
        out_len = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_index is None:
        out_index = torch.empty((B, Hkv, budget), dtype=torch.int32, device=dev)
    if out_weights is None:
        out_weights = torch.empty((B, Hkv, budget), dtype=torch.float32, device=dev)
    _check_cuda("out_len", out_len, torch.int32, (B,), dev)
    _check_cuda("out_index", out_index, torch.int32, (B, Hkv, budget), dev)
    _check_cuda("out_weights", out_weights, torch.float32, (B, Hkv, budget), dev)
    _ok(library().kv_cache_evict(
        _pack_shape(dtype, B, 1, Hkv, Hkv, D, page_size, pages, max_pages), pools[0], pools[1],
        page_table.data_ptr(), seq_len.data_ptr(), weights.data_ptr(), N, budget, recent,
        pools[2], pools[3], new_k.shape[0], new_page_table.data_ptr(), new_cols,
        out_len.data_ptr(), out_index.data_ptr(), out_weights.data_ptr(), h),
        "kv_cache_evict")
    return out_len, out_index, out_weights


# ------------------------------------------------------------------------------ 8-bit cache
def _check_codes(k_cache, v_cache, k_scale, v_scale, like):
    """Checks a cache of e4m3 codes [pages, page_size, Hkv, D] and its scales [pages, blocks, Hkv];
    returns its two pools and the slots of a block."""
    _check_strided("k_cache", k_cache, torch.float8_e4m3fn, None, like.device)
    if k_cache.ndim != 4:
        raise ValueError("k_cache must have shape [pages, page_size, Hkv, D]")
    pages, page_size, Hkv, _ = k_cache.shape
    pools = [_kv_pool("k_cache", k_cache, k_cache), _kv_pool("v_cache", v_cache, k_cache)]
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must have k_cache's shape")
    blocks = k_scale.shape[1] if k_scale.ndim == 3 else 0
    if blocks < 1 or page_size % blocks:
        raise ValueError("k_scale must have shape [pages, page_size / block, Hkv]")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is None:
            raise TypeError(f"{name} must be a CUDA tensor")
        _check_cuda(name, t, torch.float32, (pages, blocks, Hkv), like.device)
    return *pools, page_size // blocks


def kv_cache_append_q8(k, v, slots, k_cache, v_cache, k_scale, v_scale, *, stream=None):
    """Rounds new keys and values, [T, Hkv, D] or [B, P, Hkv, D] (rows one stride apart), to 8 bits
    and puts row t into slot ``slots[t]`` (int64, page * page_size + slot; -1: left out) of the pools
    k_cache and v_cache, float8_e4m3fn views [pages, page_size, Hkv, D], with scales k_scale and
    v_scale [pages, page_size / block, Hkv] fp32. All four are updated in place. Rows of one block
    stand side by side in ascending order of slots."""
    h = _raw_stream(stream, k)
    status = (_native._calls or _native.calls()).append(k, v, slots, k_cache, v_cache, k_scale,
                                                        v_scale, h)
    if status is not None:
        if status:
            raise SVError(status, "kv_cache_append_q8")
        return
    # an argument that does not fit: the checks one by one
    dtype = _KV_DTYPE.get(k.dtype)
    if dtype is None:
        raise TypeError(f"keys and values must be bfloat16 or float16, got {k.dtype}")
    if k.ndim not in (3, 4):
        raise ValueError("k must have shape [T, Hkv, D] or [B, P, Hkv, D]")
    strides = []
    for name, x in (("k", k), ("v", v)):
        _check_strided(name, x, k.dtype, k.shape, k.device)
        if x.ndim == 4 and x.shape[0] > 1 and x.shape[1] > 1 and \
                x.stride(0) != x.shape[1] * x.stride(1):
            raise ValueError(f"the rows of {name} must lie one stride apart")
        strides.append(x.stride(0) if x.ndim == 4 and x.shape[1] == 1 else x.stride(-3))
    if slots is None:
        raise TypeError("slots must be a CUDA tensor")
    _check_cuda("slots", slots, torch.int64, k.shape[:-2], k.device)
    kp, vp, block = _check_codes(k_cache, v_cache, k_scale, v_scale, k)
    pages, page_size, Hkv, D = k_cache.shape
    if k.shape[-2:] != (Hkv, D):
        raise ValueError("k must have the cache's heads and width")
    _ok(library().kv_cache_append_q8(
        _pack_shape(dtype, 1, 1, 1, Hkv, D, page_size, pages, 1), slots.numel(), k.data_ptr(),
        strides[0], k.stride(-2), v.data_ptr(), strides[1], v.stride(-2), slots.data_ptr(), kp, vp,
        k_scale.data_ptr(), v_scale.data_ptr(), block, h), "kv_cache_append_q8")


def paged_attention_q8_workspace(B: int, P: int, Hq: int, dtype, k_cache, page_table) -> int:
    pages, page_size, Hkv, D = k_cache.shape
    return int(library().paged_attention_q8_workspace(
        _pack_shape(_KV_DTYPE[dtype], B, P, Hq, Hkv, D, page_size, pages, page_table.shape[1])))


def paged_attention_q8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_len, *,
                       num_draft=None, scale=None, softcap: float = 0.0, window: int = 0,
                       slopes=None, out=None, out_lse=None, want_lse: bool = True, workspace=None,
                       stream=None):
    """paged_attention over a cache in 8 bits: k_cache and v_cache are float8_e4m3fn views [pages,
    page_size, Hkv, D] with scales k_scale and v_scale [pages, page_size / block, Hkv] fp32; q and
    out are bfloat16 or float16. Returns (out [B, P, Hq, D], lse [B, P, Hq] fp32 or None)."""
    if out is None:
        out = _made(torch.empty, q.shape, q.dtype, q.device, stream)
    if out_lse is None and want_lse:
        out_lse = _made(torch.empty, q.shape[:3], torch.float32, q.device, stream)
    h = _raw_stream(stream, q)
    ws = workspace
    if ws is None:
        ws = _ws_cache.get(("attention8", q.get_device(), h))
        if ws is not None and _capturing(h, stream):
            ws = None
    fast = (_native._calls or _native.calls()).attention8
    status = fast(q, k_cache, page_table, seq_len, num_draft, slopes, scale, softcap, window,
                  v_cache, k_scale, v_scale, out, out_lse, ws, h)
    if status is not None and status < 0 and workspace is None:
        # a first call on this stream, one that needs more than the earlier ones did, or a captured one
        ws = _workspace("attention8", -status - 1, q.device,
                        stream or torch.cuda.current_stream(q.device))
        if _ws_cache.get(("attention8", q.device, h)) is ws:
            _ws_cache["attention8", q.get_device(), h] = ws
        status = fast(q, k_cache, page_table, seq_len, num_draft, slopes, scale, softcap, window,
                      v_cache, k_scale, v_scale, out, out_lse, ws, h)
    if status is not None:
        if status:
            raise SVError(status if status > 0 else 3, "paged_attention_q8")
        return out, out_lse
    # an argument that does not fit: the checks one by one
    B, P, Hq, D = q.shape
    dev = q.device
    dtype = _KV_DTYPE.get(q.dtype)
    if dtype is None:
        raise TypeError(f"queries must be bfloat16 or float16, got {q.dtype}")
    _check_strided("q", q)
    kp, vp, block = _check_codes(k_cache, v_cache, k_scale, v_scale, q)
    pages, page_size, Hkv, d = k_cache.shape
    if d != D:
        raise ValueError("k_cache must have q's width")
    _check_cuda("page_table", page_table, torch.int32, (B, page_table.shape[-1]), dev)
    _check_cuda("seq_len", seq_len, torch.int32, (B,), dev)
    _check_cuda("num_draft", num_draft, torch.int32, (B,), dev)
    _check_cuda("slopes", slopes, torch.float32, (Hq,), dev)
    _check_cuda("out", out, q.dtype, (B, P, Hq, D), dev)
    _check_cuda("out_lse", out_lse, torch.float32, (B, P, Hq), dev)
    _check_cuda("workspace", workspace, None, None, dev)
    shape = _pack_shape(dtype, B, P, Hq, Hkv, D, page_size, pages, page_table.shape[1])
    L = library()
    if workspace is None:
        ws = _workspace("attention8", L.paged_attention_q8_workspace(shape), dev,
                        stream or torch.cuda.current_stream(dev))
    rule = _pack_rule(D ** -0.5 if scale is None else scale, softcap, window, _ptr(slopes) or 0)
    a, b, c, _ = q.stride()
    _ok(L.paged_attention_q8(
        shape, rule, q.data_ptr(), a, b, c, kp, vp, k_scale.data_ptr(), v_scale.data_ptr(), block,
        page_table.data_ptr(), seq_len.data_ptr(), _ptr(num_draft), out.data_ptr(), _ptr(out_lse),
        ws.data_ptr(), ws.numel() * ws.element_size(), h), "paged_attention_q8")
    return out, out_lse


# ------------------------------------------------------------------------------ ahead of a step
def kv_page_map(page_table, old_len, seq_len, num_new, ring, ring_state, page_size: int,
                num_pages: int, *, P: int | None = None, rows: int | None = None, out_slots=None,
                out_positions=None, out_len=None, out_first=None, out_state=None, stream=None):
    """Pages and slots of the new positions. Request r holds the pages of ``old_len`` tokens in its
    row of page_table [B, max_pages] int32 (updated in place) and is to have ``seq_len`` tokens, the
    last ``num_new`` of them new: it takes the pages it lacks from the front of ``ring`` (int32, the
    free pages, updated in place; ``ring_state`` [2] int32 holds the first one's place and how many
    there are) or gives pages back to its end. Rows are [B, P], or packed in ``rows`` rows (of
    ``out_slots``, where that is given).
    Returns (slots [B, P] or [rows] int64, positions int32 likewise, both -1 in rows of no new
    token; out_len [B] int32: seq_len, old_len where no pages were left, -1 for a data error;
    first rows [B + 1] int32; the ring's new state [2] int32, also of a batch without requests)."""
    if out_slots is None:
        if (P is None) == (rows is None):
            raise ValueError("give P (rows per request) or rows (packed)")
        size = (page_table.shape[0], P) if rows is None else (rows,)
        out_slots = _made(torch.empty, size, torch.int64, page_table.device, stream)
    elif (P is not None and (out_slots.ndim != 2 or out_slots.shape[1] != P)
          or rows is not None and (out_slots.ndim != 1 or out_slots.shape[0] != rows)):
        raise ValueError(f"out_slots of shape {tuple(out_slots.shape)} is not of P={P}, rows={rows}")
    B = page_table.shape[0]
    made = [_made(torch.empty, size, torch.int32, page_table.device, stream) if t is None else t
            for t, size in ((out_positions, out_slots.shape), (out_len, (B,)),
                            (out_first, (B + 1,)), (out_state, (2,)))]
    h = _raw_stream(stream, page_table)
    status = (_native._calls or _native.calls()).page_map(
        page_table, old_len, seq_len, num_new, ring, ring_state, page_size, num_pages, out_slots,
        *made, h)
    if status is not None:
        if status:
            raise SVError(status, "kv_page_map")
        return out_slots, *made
    # an argument that does not fit: the checks one by one
    dev = page_table.device
    padded = out_slots.ndim == 2
    if out_slots.ndim not in (1, 2) or padded and (out_slots.shape[0] != B or out_slots.shape[1] < 1):
        raise ValueError("slots must have shape [B, P] or [rows]")
    for name, t, dtype, shape in (
            ("page_table", page_table, torch.int32, (B, page_table.shape[-1])),
            ("old_len", old_len, torch.int32, (B,)), ("seq_len", seq_len, torch.int32, (B,)),
            ("num_new", num_new, torch.int32, (B,)), ("ring", ring, torch.int32, (ring.numel(),)),
            ("ring_state", ring_state, torch.int32, (2,)),
            ("out_slots", out_slots, torch.int64, out_slots.shape),
            ("out_positions", made[0], torch.int32, out_slots.shape),
            ("out_len", made[1], torch.int32, (B,)), ("out_first", made[2], torch.int32, (B + 1,)),
            ("out_state", made[3], torch.int32, (2,))):
        if t is None:
            raise TypeError(f"{name} must be a CUDA tensor")
        _check_cuda(name, t, dtype, shape, dev)
    for name, x in (("page_size", page_size), ("num_pages", num_pages), ("rows", out_slots.numel()),
                    ("the ring's size", ring.numel())):
        if not -2 ** 31 <= x < 2 ** 31:  # (what ctypes would cut to 32 bits)
            raise ValueError(f"{name} is {x}, past 32 bits")
    _ok(library().kv_page_map(
        B, page_size, num_pages, page_table.data_ptr(), page_table.shape[1], old_len.data_ptr(),
        seq_len.data_ptr(), num_new.data_ptr(), ring.data_ptr(), ring.numel(),
        ring_state.data_ptr(), out_slots.shape[1] if padded else 0, out_slots.numel(),
        out_slots.data_ptr(), *(t.data_ptr() for t in made), h), "kv_page_map")
    return out_slots, *made


def qk_norm_rotate(q, k, positions, inv_freq=None, *, q_weight=None, k_weight=None,
                   eps: float = 1e-6, norm: bool = True, interleaved: bool = False, out_q=None,
                   out_k=None, stream=None):
    """Divides every head of q [..., Hq, D] and k [..., Hkv, D] by its root mean square, multiplies
    by the weights [D] (fp32 or q's type), and rotates its first 2 * len(inv_freq) components by
    position * inv_freq (fp32 or fp64): component i with i + R/2, or 2i with 2i + 1 where
    ``interleaved``. ``positions`` [...] int32; rows at a negative one are left as they are (in outputs that
    the call makes, as the memory was).
    Returns (out_q, out_k), which may be q and k themselves."""
    if out_q is None:
        out_q = _made(torch.empty, q.shape, q.dtype, q.device, stream)
    if out_k is None:
        out_k = _made(torch.empty, k.shape, k.dtype, k.device, stream)
    h = _raw_stream(stream, q)
    status = (_native._calls or _native.calls()).rotate(
        q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, norm, out_q, out_k, h)
    if status is not None:
        if status:
            raise SVError(status, "qk_norm_rotate")
        return out_q, out_k
    # an argument that does not fit: the checks one by one
    dtype = _KV_DTYPE.get(q.dtype)
    if dtype is None:
        raise TypeError(f"queries must be bfloat16 or float16, got {q.dtype}")
    if q.ndim not in (3, 4) or k.ndim != q.ndim:
        raise ValueError("q and k must have shape [T, heads, D] or [B, P, heads, D]")
    lead, D, dev = q.shape[:-2], q.shape[-1], q.device
    _check_strided("q", q)
    _check_strided("k", k, q.dtype, (*lead, k.shape[-2], D), dev)
    _check_strided("out_q", out_q, q.dtype, q.shape, dev)
    _check_strided("out_k", out_k, q.dtype, k.shape, dev)
    if positions is None:
        raise TypeError("positions must be a CUDA tensor")
    _check_cuda("positions", positions, torch.int32, lead, dev)
    wide = inv_freq is not None and inv_freq.dtype == torch.float64
    half = 0 if inv_freq is None else inv_freq.numel()
    _check_cuda("inv_freq", inv_freq, torch.float64 if wide else torch.float32, (half,), dev)
    w = q_weight if q_weight is not None else k_weight
    w32 = w is not None and w.dtype == torch.float32
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        _check_cuda(name, t, torch.float32 if w32 else q.dtype, (D,), dev)
    rows = []
    for x, out, weight in ((q, out_q, q_weight), (k, out_k, k_weight)):
        rows.append(_native.HeadRows(
            x.data_ptr(), x.stride(0) if x.ndim == 4 else 0, x.stride(-3), x.stride(-2),
            out.data_ptr(), out.stride(0) if x.ndim == 4 else 0, out.stride(-3), out.stride(-2),
            x.shape[-2], _ptr(weight)))
    _ok(library().qk_norm_rotate(
        dtype, lead[0] if q.ndim == 4 else 1, lead[-1], D, 2 * half, ctypes.byref(rows[0]),
        ctypes.byref(rows[1]), int(w32), positions.data_ptr(), _ptr(inv_freq), int(wide),
        int(bool(norm)), float(eps), int(bool(interleaved)), h), "qk_norm_rotate")
    return out_q, out_k
