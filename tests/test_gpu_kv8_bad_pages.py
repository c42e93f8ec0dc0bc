"""Pages outside the pool in a long work list of short requests over a cache in 8 bits."""
import pytest
import torch

import kv8_reference as ref8
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,G,P", [(64, 8, 3), (64, 8, 6), (64, 8, 8), (64, 4, 1), (64, 4, 4), (128, 4, 1),
                                   (128, 8, 3), (256, 2, 1)])
def test_bad_pages_in_a_work_list_of_short_requests(dtype, D, G, P):
    """Every piece is one tile and a CTA walks twenty or more: the rows of a request whose first page is
    none are NaN, all of them, and the others keep their bits."""
    B, Hkv, page = 400, 16, 16
    g = torch.Generator().manual_seed(D + G + P)
    lens = torch.randint(P, 129, (B,), generator=g)
    counts = (-(-lens // page)).tolist()
    table, at = torch.full((B, 8), -1, dtype=torch.int32), 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.arange(at, at + c)
        at += c
    dg = torch.Generator(device="cuda").manual_seed(1)
    codes = [torch.randn((at, page, Hkv, D), generator=dg, device="cuda").mul(64).clamp(-448, 448).to(ref8.CODE)
             for _ in range(2)]
    scales = [torch.full((at, 1, Hkv), 2.0 ** -6, device="cuda") for _ in range(2)]
    q = torch.randn((B, P, Hkv * G, D), generator=dg, device="cuda").to(dtype)
    good, good_lse = sv.paged_attention_q8(q, *codes, *scales, table.cuda(), lens.int().cuda())
    assert bool(good.isfinite().all()) and bool(good_lse.isfinite().all())
    for share in (1.0, 0.9, 0.3):
        bad = torch.rand(B, generator=g) < share
        wrong = table.clone()
        wrong[bad, 0] = torch.where(torch.arange(int(bad.sum())) % 2 == 0, -1, at).int()
        wrong = wrong.cuda()
        for _ in range(5):
            out, lse = sv.paged_attention_q8(q, *codes, *scales, wrong, lens.int().cuda())
            torch.cuda.synchronize()
            assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
            assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], good_lse[~bad])
