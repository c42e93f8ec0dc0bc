"""Outputs of the calls around a cache in 8 bits that share memory with one another or with what is read:
refused on the host (no GPU: every call here returns before any CUDA call)."""
import ctypes

import pytest

import speculative_decoding_verification_17_gb300 as sv
from speculative_decoding_verification_17_gb300 import _native

INVALID = 1


def pool(data, page=4096, token=256, head=128):
    return ctypes.byref(_native.KvPool(data, page, token, head))


def append(pages=40, Hkv=2, **kw):
    """40 pages of 16 slots and 2 heads of 128, a scale per 16 slots: 320 bytes of scales."""
    a = dict(shape=ctypes.byref(_native.KvShape(1, 2, 3, 8, Hkv, 128, 16, pages, 10)), rows=5, k=0x10000, kr=256,
             kh=128, v=0x18000, vr=256, vh=128, slots=0x1f000, kp=pool(0x20000), vp=pool(0x80000), ks=0x100000,
             vs=0x110000, block=16, st=None)
    a.update(kw)
    return sv.library().kv_cache_append_q8(*a.values())


@pytest.mark.parametrize("kw", [
    dict(vp=pool(0x20000)), dict(kp=pool(0x80000)), dict(vp=pool(0x20000, page=8192)),
    dict(vs=0x100000), dict(vs=0x100000 + 316), dict(vs=0x100000 - 316), dict(ks=0x110000 + 4),
    dict(kp=pool(0x20000, token=64)), dict(vp=pool(0x80000, head=64)), dict(kp=pool(0x20000, page=112)),
    dict(pages=1, Hkv=1, vp=pool(0x80000, page=16, head=16, token=112)),
])
def test_pools_and_scales_that_share_memory_are_refused(kw):
    assert append(**kw) == INVALID


def rows(data, out, heads=4, req=1024, row=512, head=128, oq=1024, orow=512, oh=128):
    return ctypes.byref(_native.HeadRows(data, req, row, head, out, oq, orow, oh, heads, None))


Q, K = (0x100000, 0x200000), (0x300000, 0x400000)  # data, out


def rotate(q, k, B=3, P=2):
    return sv.library().qk_norm_rotate(1, B, P, 128, 128, q, k, 1, 0x500000, 0x600000, 0, 1, 1e-6, 0, None)


@pytest.mark.parametrize("q,k", [
    (rows(Q[0], Q[1]), rows(K[0], Q[1], heads=1)),  # one place for both results
    (rows(Q[0], K[0]), rows(K[0], K[1], heads=1)),  # the keys under the queries' result
    (rows(Q[0], Q[1]), rows(K[0], Q[0], heads=1)),
    (rows(Q[0], Q[0], oq=2048), rows(*K)),          # in place, but elsewhere
    (rows(Q[0], Q[0], orow=256, oq=4096), rows(*K)),
    (rows(*Q), rows(K[0], K[0], head=256, row=1024, req=2048)),
    (rows(Q[0], Q[1], oh=64), rows(*K)),            # heads that overlap
    (rows(*Q), rows(K[0], K[1], orow=120)),
    (rows(*Q), rows(K[0], K[1], oq=8)),
])
def test_rows_that_share_memory_are_refused(q, k):
    assert rotate(q, k) == INVALID
