"""paged_attention and attention_weight_sum over batches in which long caches are followed by runs of
requests without work for the tensor cores (padding slots of length 0, counts out of range, no row
that counts): more of them in one CTA's range than its queue of pieces holds."""
import math

import pytest
import torch

import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def batch(Hkv, G, P, D, page, groups, long, dtype=torch.bfloat16):
    """`groups` times [a long cache, an empty one, one with bad counts, a short one]."""
    g = torch.Generator().manual_seed(Hkv + D)
    lens, nd, bad = [], [], []
    for i in range(groups):
        lens += [long - int(torch.randint(0, 300, (1,), generator=g)), 0, 5, 1 + i % 3]
        nd += [P - 1, i % P, P - 1, min(i % 3, P - 1)]
        bad += [False, False, True, False]
    B = len(lens)
    lens, nd = torch.tensor(lens).int(), torch.tensor(nd).int()
    cols = -(-long // page)
    total = int((-(-lens.long() // page)).sum())
    ids, table, at = torch.randperm(total, generator=g).int(), torch.full((B, cols), -1).int(), 0
    for b, c in enumerate((-(-lens.long() // page)).tolist()):
        table[b, :c] = ids[at:at + c]
        at += c
    dg = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((total, page, Hkv, D), generator=dg, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((B, P, Hkv * G, D), generator=dg, device="cuda").to(dtype)
    bad = torch.tensor(bad)
    said = lens.clone()
    said[bad] = torch.tensor([-3, cols * page + 1])[torch.arange(int(bad.sum())) % 2].int()
    return q, k, v, table.cuda(), lens.cuda(), said.cuda(), nd.cuda(), bad.cuda()


SHAPES = [(8, 4, 1, 128, 64, 24, 8000), (16, 2, 2, 64, 16, 24, 4000), (16, 4, 5, 128, 32, 16, 6000),
          (16, 8, 9, 128, 128, 12, 6000), (16, 2, 3, 256, 64, 16, 5000)]


@pytest.mark.parametrize("Hkv,G,P,D,page,groups,long", SHAPES)
def test_attention_beside_runs_of_empty_requests(Hkv, G, P, D, page, groups, long):
    q, k, v, table, lens, said, nd, bad = batch(Hkv, G, P, D, page, groups, long)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    for _ in range(2):
        sv.paged_attention(q, k, v, table, said, num_draft=nd, out=out, out_lse=lse)
    torch.cuda.synchronize()
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    want, want_lse, tol, tol_lse, live = ref.attention_on_device(q, k, v, table, lens, nd,
                                                                 scale=D ** -0.5)
    fine = live & ~bad[:, None]
    assert ref.close(out[fine], want[fine], tol[fine])
    assert ref.close(lse[fine], want_lse[fine], tol_lse[fine])
    rest = ~live & ~bad[:, None]
    assert bool((out[rest] == 7).all()) and bool((lse[rest] == 7).all())
    # the row of an empty cache sees nothing
    empty = fine & (lens == 0)[:, None]
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())


@pytest.mark.parametrize("Hkv,G,P,D,page,groups,long", SHAPES)
@pytest.mark.parametrize("prior", [False, True])
def test_key_weights_beside_requests_without_rows(Hkv, G, P, D, page, groups, long, prior):
    q, k, v, table, lens, said, nd, bad = batch(Hkv, G, P, D, page, groups, long)
    _, lse = sv.paged_attention(q, k, v, table, said, num_draft=nd)
    acc = nd.clone()
    acc[(torch.arange(len(lens), device="cuda") % 8) == 4] = -1  # long caches without a row
    acc[lens == 0] = -1
    N = int(lens.max()) + 3
    before = torch.rand((len(lens), Hkv, N), device="cuda")
    out = before.clone() if prior else torch.full_like(before, 7.0)
    sv.attention_weight_sum(q, k, table, said, lse, num_draft=nd, accept_len=acc,
                            prior=out if prior else None, out=out)
    torch.cuda.synchronize()
    held = before if prior else torch.zeros_like(before)
    inside = (torch.arange(N, device="cuda") < lens[:, None])[:, None].expand_as(out)
    b = torch.nonzero(bad).flatten()
    # every `long` and `P` here gives the bad requests lengths out of range
    assert bool(out[b, :, 0].isnan().all())
    kept = before if prior else torch.full_like(before, 7.0)
    assert torch.equal(out[b, :, 1:], kept[b, :, 1:])
    fine = ~bad
    assert torch.equal(out[~inside & fine[:, None, None]], kept[~inside & fine[:, None, None]])
    none = fine & (acc < 0)
    assert torch.equal(out[none][inside[none]], held[none][inside[none]])
    # every row that counts and sees a key gave 1 per head in all
    rows = torch.arange(P, device="cuda")
    gave = ((rows <= acc[:, None]) & (lens[:, None] - 1 - nd[:, None] + rows >= 0)).sum(1) * G
    got = torch.where(inside, out.double() - held.double(), 0.0).sum(-1)[fine]
    # (a sum of up to 8000 fp32 values below 2: half steps of 2^-24 each, and the weights' 2e-4)
    assert torch.allclose(got, gave[fine, None].double().expand_as(got), rtol=2e-4, atol=1e-3)


def test_key_weights_of_blocks_of_rows_that_see_nothing():
    """Rows in several passes over the keys, of which the first sees no key at all."""
    Hkv, G, P, D = 2, 64, 17, 64
    lens = torch.tensor([3, 40, 3, 9]).int().cuda()
    nd = torch.tensor([16, 16, 5, 16]).int().cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((4, P, Hkv * G, D), generator=g, device="cuda").bfloat16()
    k, v = (torch.randn((16, 16, Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(16, device="cuda").int().view(4, 4)
    _, lse = sv.paged_attention(q, k, v, table, lens, num_draft=nd)
    prior = torch.rand((4, Hkv, 64), device="cuda")
    out = sv.attention_weight_sum(q, k, table, lens, lse, num_draft=nd, prior=prior,
                                  out=torch.full_like(prior, 7.0))
    rows = torch.arange(P, device="cuda")
    gave = ((rows <= nd[:, None]) & (lens[:, None] - 1 - nd[:, None] + rows >= 0)).sum(1) * G
    inside = (torch.arange(64, device="cuda") < lens[:, None])[:, None].expand_as(out)
    got = torch.where(inside, out.double() - prior.double(), 0.0).sum(-1)
    assert torch.allclose(got, gave[:, None].double().expand_as(got), rtol=2e-4, atol=1e-3)
    assert bool((out[~inside] == 7).all())
