"""Arguments of kv_page_map that contradict one another, or that 32 bits do not hold."""
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import speculative_decoding_verification_17_gb300 as sv


@pytest.mark.parametrize("size,kw", [
    ((3, 4), dict(P=5)), ((3, 4), dict(rows=12)), ((12,), dict(rows=13)), ((12,), dict(P=4)),
    ((3, 4), dict(P=4, rows=12)), ((12,), dict(P=4, rows=12)),
])
def test_rows_that_out_slots_does_not_have(size, kw):
    if torch.cuda.is_available():
        pytest.skip("fakes stand in for the tensors of a GPU")
    with FakeTensorMode():
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        slots = torch.empty(size, dtype=torch.int64, device="cuda")
        with pytest.raises(ValueError, match="out_slots"):
            sv.kv_page_map(i32(3, 6), i32(3), i32(3), i32(3), i32(9), i32(2), 16, 9, out_slots=slots, **kw,
                           stream=SimpleNamespace(cuda_stream=0))


@pytest.mark.parametrize("page,pages,ring,rows", [
    (2 ** 32 + 16, 9, 9, 12), (16, 2 ** 32 + 9, 9, 12), (16, 9, 2 ** 32 + 9, 12), (16, 9, 9, 2 ** 32 + 12),
])
def test_sizes_past_32_bits(page, pages, ring, rows):
    """ctypes cuts them to their lower bits, which are sizes like any other."""
    if torch.cuda.is_available():
        pytest.skip("fakes stand in for the tensors of a GPU")
    with FakeTensorMode():
        i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        with pytest.raises(ValueError, match="32 bits"):
            sv.kv_page_map(i32(3, 6), i32(3), i32(3), i32(3), i32(ring), i32(2), page, pages, out_slots=slots,
                           out_positions=i32(rows), out_len=i32(3), out_first=i32(4), out_state=i32(2),
                           stream=SimpleNamespace(cuda_stream=0))
