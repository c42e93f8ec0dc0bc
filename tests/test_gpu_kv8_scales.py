"""paged_attention_q8 of fp16 queries over value scales far apart."""
import pytest
import torch

import kv8_reference as ref8
import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("spread,plain", [(4.0, True), (8.0, False), (20.0, False)])
@pytest.mark.parametrize("D,G,P", [(64, 4, 3), (128, 4, 3), (128, 4, 1), (256, 4, 5)])
def test_value_scales_far_apart_beside_fp16_queries(spread, plain, D, G, P):
    """Blocks whose values are millions of times smaller than others', with outputs that fp16 holds."""
    cache = ref8.Cache8([700, 31, 1500], 32, 8, 2, D, seed=4, spread=spread, plain_scales=plain)
    cache.scales[0].clamp_(2.0 ** -9, 2.0 ** -5)
    cache.scales[1].clamp_(2.0 ** -39, 2.0 ** 4)
    q = torch.randn((3, P, 2 * G, D), generator=torch.Generator().manual_seed(D)).half()
    nd = [P - 1, min(1, P - 1), 0]
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    sv.paged_attention_q8(q.cuda(), cache.view(0, "cuda"), cache.view(1, "cuda"), cache.scales[0].cuda(),
                          cache.scales[1].cuda(), cache.table.cuda(), cache.seq_len.cuda(), num_draft=i32(nd),
                          out=out, out_lse=lse)
    want, want_lse, tol, tol_lse = ref8.attention8(cache, q, nd, scale=D ** -0.5)
    live = torch.arange(P) <= torch.tensor(nd)[:, None]
    assert ref.close(lse.cpu()[live], want_lse[live], tol_lse[live])
    assert ref.close(out.cpu()[live], want[live], tol[live])
