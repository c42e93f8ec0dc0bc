"""paged_attention_q8's bounded waits do run out."""
import ctypes

import pytest
import torch

import kv8_reference as ref8
import speculative_decoding_verification_17_gb300 as sv
from speculative_decoding_verification_17_gb300 import _native

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,P,page,block,dtype", [
    (128, 4, 1, 64, 64, torch.bfloat16), (128, 8, 6, 16, 16, torch.float16),
    (64, 8, 9, 32, 8, torch.bfloat16), (256, 2, 3, 128, 32, torch.bfloat16)])
def test_waits_run_out_at_the_smallest_limit(D, G, P, page, block, dtype):
    """A first copy takes longer than a microsecond to land: some rows are NaN, the rest as they are."""
    B, Hkv = 30, 2
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(100, 6000, (B,), generator=g).tolist()
    cache = ref8.Cache8(lens, page, block, Hkv, D, seed=2)
    q = torch.randn((B, P, Hkv * G, D), generator=g).to(dtype).cuda()
    k, v, ks, vs = cache.view(0, "cuda"), cache.view(1, "cuda"), cache.scales[0].cuda(), cache.scales[1].cuda()
    table, n = cache.table.cuda(), cache.seq_len.cuda()
    want, want_lse = sv.paged_attention_q8(q, k, v, ks, vs, table, n)
    shape = _native.KvShape(1 if dtype == torch.bfloat16 else 2, B, P, Hkv * G, Hkv, D, page, k.shape[0],
                            table.shape[1])
    rule = _native.ScoreRule(D ** -0.5, 0.0, 0, None)
    pool = lambda t: ctypes.byref(_native.KvPool(t.data_ptr(), *t.stride()[:3]))  # noqa: E731
    L = sv.library()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    ws = torch.zeros(L.paged_attention_q8_workspace(ctypes.byref(shape)), dtype=torch.uint8, device="cuda")
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(1)  # the codes are no longer in L2
    torch.cuda.synchronize()
    status = L.paged_attention_q8_wait_selftest(
        ctypes.byref(shape), ctypes.byref(rule), q.data_ptr(), *q.stride()[:3], pool(k), pool(v),
        ks.data_ptr(), vs.data_ptr(), block, table.data_ptr(), n.data_ptr(), None, out.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.numel(), 1, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()
    gone = out.isnan().all(-1) & lse.isnan()
    same = (out == want).all(-1) & (lse == want_lse)
    assert bool((gone | same).all()) and bool(gone.any())
