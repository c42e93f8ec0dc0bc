"""The bounded waits of paged_attention and attention_weight_sum, driven to their limit: the calls end
on their own, and what they owe is either what the ordinary call gives or NaN, never what the output
or the workspace held before."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_17_gb300 as sv
from speculative_decoding_verification_17_gb300 import _native

INVALID = 1


def test_the_limit_is_checked():
    L = sv.library()
    for us in (0, 100001):
        assert L.paged_attention_wait_selftest(*[None] * 3, 0, 0, 0, *[None] * 8, 0, us, None) == INVALID
        assert L.attention_weight_sum_wait_selftest(
            *[None] * 3, 0, 0, 0, *[None] * 5, 0, 0, 0, None, None, None, 0, us, None) == INVALID


def case(Hkv, G, P, D, page, dtype, seed=0):
    """Long caches, empty ones and ones with bad counts."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 6000, (40,), generator=g).int()
    lens[::5], lens[2] = 0, 9000
    nd = torch.randint(0, P, (40,), generator=g).int()
    counts = -(-lens.long() // page)
    cols, total = int(counts.max()), int(counts.sum())
    ids, table, at = torch.randperm(total, generator=g).int(), torch.full((40, cols), -1).int(), 0
    for b, c in enumerate(counts.tolist()):
        table[b, :c] = ids[at:at + c]
        at += c
    lens[7], nd[8] = -1, P
    dg = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn((total, page, Hkv, D), generator=dg, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((40, P, Hkv * G, D), generator=dg, device="cuda").to(dtype)
    return q, k, v, table.cuda(), lens.cuda(), nd.cuda()


def common(q, k, table):
    B, P, Hq, D = q.shape
    shape = _native.KvShape(1 if q.dtype == torch.bfloat16 else 2, B, P, Hq, k.shape[2], D,
                            k.shape[1], k.shape[0], table.shape[1])
    rule = _native.ScoreRule(D ** -0.5, 0.0, 0, None)
    pool = lambda t: ctypes.byref(_native.KvPool(t.data_ptr(), *t.stride()[:3]))  # noqa: E731
    return ctypes.byref(shape), ctypes.byref(rule), q.data_ptr(), *q.stride()[:3], pool


SHAPES = [(4, 4, 1, 128, 64, torch.bfloat16), (2, 8, 6, 128, 16, torch.float16),
          (2, 8, 9, 64, 32, torch.bfloat16), (4, 2, 3, 256, 128, torch.bfloat16)]


@pytest.mark.gpu
@pytest.mark.parametrize("us", [1, 2, 4, 10, 40])
@pytest.mark.parametrize("Hkv,G,P,D,page,dtype", SHAPES)
def test_rows_of_a_cta_that_gives_up_are_nan(Hkv, G, P, D, page, dtype, us):
    q, k, v, table, lens, nd = case(Hkv, G, P, D, page, dtype)
    want, want_lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    sv.paged_attention(q, k, v, table, lens, num_draft=nd, out=want, out_lse=want_lse)
    *head, pool = common(q, k, table)
    ws = torch.zeros(sv.paged_attention_workspace(*q.shape[:3], k, table), dtype=torch.uint8,
                     device="cuda")
    # (a first ordinary call leaves finite parts in the workspace)
    sv.paged_attention(q, k, v, table, lens, num_draft=nd, workspace=ws)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    assert sv.library().paged_attention_wait_selftest(
        *head, pool(k), pool(v), table.data_ptr(), lens.data_ptr(), nd.data_ptr(), out.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.numel(), us, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    gone = out.isnan().all(-1) & lse.isnan()
    same = ((out == want) | (out.isnan() & want.isnan())).all(-1)
    same &= (lse == want_lse) | (lse.isnan() & want_lse.isnan())
    assert bool((gone | same).all())
    rows = torch.arange(P, device="cuda")
    dead = (rows > nd[:, None])[..., None].expand_as(lse) & ((lens >= 0) & (nd < P))[:, None, None]
    assert bool((out[dead] == 7).all()) and bool((lse[dead] == 7).all())
    if us == 1:  # (a first copy takes longer than that to land)
        assert bool((gone & ~want_lse.isnan()).any())
    # the device and the workspace serve an ordinary call
    sv.paged_attention(q, k, v, table, lens, num_draft=nd, out=out, out_lse=lse, workspace=ws)
    assert torch.equal(out.nan_to_num(5.0), want.nan_to_num(5.0))
    assert torch.equal(lse.nan_to_num(5.0), want_lse.nan_to_num(5.0))


@pytest.mark.gpu
@pytest.mark.parametrize("us", [1, 2, 4, 10, 40])
@pytest.mark.parametrize("Hkv,G,P,D,page,dtype", SHAPES)
def test_key_weights_of_a_cta_that_gives_up_are_nan(Hkv, G, P, D, page, dtype, us):
    q, k, v, table, lens, nd = case(Hkv, G, P, D, page, dtype, seed=1)
    _, lse = sv.paged_attention(q, k, v, table, lens, num_draft=nd)
    N = table.shape[1] * page
    prior = torch.rand((40, Hkv, N), device="cuda")
    want, out = torch.full_like(prior, 7.0), torch.full_like(prior, 7.0)
    sv.attention_weight_sum(q, k, table, lens, lse, num_draft=nd, prior=prior, out=want)
    *head, pool = common(q, k, table)
    assert sv.library().attention_weight_sum_wait_selftest(
        *head, pool(k), table.data_ptr(), lens.data_ptr(), nd.data_ptr(), lse.data_ptr(),
        *lse.stride(), None, prior.data_ptr(), out.data_ptr(), N, us,
        torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    inside = (torch.arange(N, device="cuda") < lens[:, None])[:, None].expand_as(out)
    assert bool(((out == want) | out.isnan()).all())
    first = torch.zeros_like(inside)
    first[:, :, 0] = True
    assert bool((out[~inside & ~first] == 7).all())  # (bad counts: NaN in slot 0)
    if us == 1:
        assert bool((out.isnan() & ~want.isnan()).any())
    sv.attention_weight_sum(q, k, table, lens, lse, num_draft=nd, prior=prior, out=out)
    assert torch.equal(out.nan_to_num(5.0), want.nan_to_num(5.0))
