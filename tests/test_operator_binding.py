"""What the binding of the calls around the verify does with arguments that are no ordinary CUDA
tensors. No GPU: the tensors are fake, and every call raises before it launches anything."""
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import speculative_decoding_verification_17_gb300 as sv

STREAM = SimpleNamespace(cuda_stream=0)


@pytest.fixture
def fake():
    if torch.cuda.is_available():
        pytest.skip("fakes stand in for the tensors of a GPU")
    with FakeTensorMode(allow_non_fake_inputs=True):
        yield lambda *s, dtype=torch.bfloat16, device="cuda": torch.empty(s, dtype=dtype, device=device)


def calls(new):
    """name -> (the call as a function of its first tensor, that tensor's sizes)."""
    i32 = lambda *s: new(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: new(*s, dtype=torch.float32)  # noqa: E731
    k, table, n = new(4, 16, 1, 64), i32(1, 4), i32(1)
    return {
        "logit_adjust": (lambda z: sv.logit_adjust(z, out=new(1, 1, 64), stream=STREAM), (1, 1, 64)),
        "paged_attention": (lambda q: sv.paged_attention(
            q, k, k, table, n, out=new(1, 1, 2, 64), out_lse=f32(1, 1, 2), stream=STREAM),
            (1, 1, 2, 64)),
        "attention_weight_sum": (lambda q: sv.attention_weight_sum(
            q, k, table, n, f32(1, 1, 2), out=f32(1, 1, 64), stream=STREAM), (1, 1, 2, 64)),
        "kv_cache_evict": (lambda c: sv.kv_cache_evict(
            c, c, table, n, f32(1, 1, 64), 16, 0, c, c, table, out_len=i32(1),
            out_index=i32(1, 1, 16), out_weights=f32(1, 1, 16), stream=STREAM), (4, 16, 1, 64)),
    }


NAMES = ["logit_adjust", "paged_attention", "attention_weight_sum", "kv_cache_evict"]


@pytest.mark.parametrize("name", NAMES)
def test_a_transformed_tensor_is_refused(fake, name):
    """A tensor inside torch.func.vmap has no address: an error, not the end of the process."""
    fn, sizes = calls(fake)[name]
    with pytest.raises((RuntimeError, TypeError, ValueError)):
        torch.func.vmap(fn)(fake(2, *sizes))


@pytest.mark.parametrize("workspace", [dict(device="cpu", dtype=torch.uint8), "strided", "text"])
def test_a_workspace_off_the_device_is_refused(fake, workspace):
    """Its address would be written by the kernel."""
    k, table, n = fake(4, 16, 1, 64), fake(1, 4, dtype=torch.int32), fake(1, dtype=torch.int32)
    if workspace == "strided":
        ws = fake(1 << 21, 8, dtype=torch.uint8)[:, 0]
    elif workspace == "text":
        ws = "workspace"
    else:
        ws = fake(1 << 24, **workspace)
    with pytest.raises((TypeError, ValueError)):
        sv.paged_attention(fake(1, 1, 2, 64), k, k, table, n, out=fake(1, 1, 2, 64),
                           out_lse=fake(1, 1, 2, dtype=torch.float32), workspace=ws, stream=STREAM)
