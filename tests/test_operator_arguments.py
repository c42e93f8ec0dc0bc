"""Refusals of kv_cache_evict and its binding that come before anything is launched or made (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode

import speculative_decoding_verification_17_gb300 as sv
from speculative_decoding_verification_17_gb300 import _native

INVALID = 1


def evict(**kw):
    """2 requests of 2 heads, tables of 10 and 3 pages of 16, every array in a place of its own."""
    shape = ctypes.byref(_native.KvShape(1, 2, 1, 2, 2, 128, 16, 40, 10))
    pool = lambda at: ctypes.byref(_native.KvPool(at, 4096, 256, 128))  # noqa: E731
    a = dict(k=pool(0x100000), v=pool(0x200000), table=0x300000, lens=0x310000, w=0x320000,
             stride=160, budget=40, recent=8, nk=pool(0x400000), nv=pool(0x500000), npages=20,
             ntable=0x600000, ncols=3, ol=0x610000, oi=0x620000, ow=0x630000, st=None)
    a.update(kw)
    return sv.library().kv_cache_evict(shape, *a.values())


@pytest.mark.parametrize("kw", [
    dict(ol=0x310000), dict(ol=0x310004), dict(ol=0x30fffc), dict(ow=0x320000),
    dict(ow=0x320000 + 4 * (2 * 2 * 160 - 1)), dict(ow=0x320000 - 4 * (2 * 2 * 40 - 1)),
])
def test_outputs_over_what_is_read_are_refused(kw):
    """In place, one head's CTA would overwrite what another still reads."""
    assert evict(**kw) == INVALID


class NothingMade(TorchDispatchMode):
    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        assert "empty" not in str(func) and "zeros" not in str(func), func
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("budget", [0, -1, 65, 10 ** 9, 2 ** 31 - 1])
def test_a_budget_its_pages_cannot_hold_makes_no_outputs(budget, monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("fakes stand in for the tensors of a GPU")
    monkeypatch.setattr(sv, "_raw_stream", lambda stream, like: 0)
    with FakeTensorMode():
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        kv, table, n = new(4, 16, 2, 64), new(1, 4, dtype=torch.int32), new(1, dtype=torch.int32)
        w, length = new(1, 2, 64, dtype=torch.float32), new(1, dtype=torch.int32)
        with NothingMade(), pytest.raises(sv.SVError) as e:
            sv.kv_cache_evict(kv, kv, table, n, w, budget, 0, kv, kv, table, out_len=length)
        assert e.value.status == INVALID


@pytest.mark.parametrize("make", [int, np.int64, np.int32])
def test_integers_of_numpy_take_the_short_way(make):
    if torch.cuda.is_available():
        pytest.skip("fakes stand in for the tensors of a GPU")
    with FakeTensorMode():
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        kv, table, n = new(4, 16, 2, 64), new(1, 4, dtype=torch.int32), new(1, dtype=torch.int32)
        made = _native.calls().evict(kv, kv, table, n, new(1, 2, 64, dtype=torch.float32), make(65),
                                     make(0), kv, kv, table, None, None, None, 0)
    assert made == (INVALID, None, None, None)  # (judged, not handed to the slow checks)
