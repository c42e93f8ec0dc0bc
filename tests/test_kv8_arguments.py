"""Arguments of kv_page_map that contradict one another."""
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
