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
