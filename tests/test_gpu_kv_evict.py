"""kv_cache_evict against a sort: ties, NaN and infinities among the weights, budgets around the
length, pages of every kind, bad tables, and the same pool as source and destination."""
import math

import pytest
import torch

import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def weights_of(B, Hkv, N, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "random":
        return torch.randn((B, Hkv, N), generator=g)
    if kind == "ties":
        return torch.randint(0, 3, (B, Hkv, N), generator=g).float()
    if kind == "equal":
        return torch.zeros((B, Hkv, N))
    special = torch.tensor([math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42, 1.0])
    return special[torch.randint(0, 8, (B, Hkv, N), generator=g)]


def run(cache, w, budget, recent, *, order="token", same_pool=False, stream=None):
    B, Hkv, page = w.shape[0], w.shape[1], cache.page
    k, v = cache.view(0, "cuda"), cache.view(1, "cuda")
    cols = -(-budget // page)
    pages = B * cols + 2
    perm = torch.randperm(pages)[:B * cols].view(B, cols).int()
    if same_pool:
        off = k.shape[0]
        k = torch.cat([k, torch.full((pages, *k.shape[1:]), 7.0, dtype=k.dtype, device="cuda")])
        v = torch.cat([v, torch.full((pages, *v.shape[1:]), 7.0, dtype=v.dtype, device="cuda")])
        nk, nv, perm = k, v, perm + off
    else:
        shape = (pages, page, Hkv, cache.D) if order == "token" else (pages, Hkv, page, cache.D)
        nk, nv = (torch.full(shape, 7.0, dtype=k.dtype, device="cuda") for _ in range(2))
        if order == "head":
            nk, nv = nk.transpose(1, 2), nv.transpose(1, 2)
    got = sv.kv_cache_evict(k, v, cache.table.cuda(), cache.seq_len.cuda(), w.cuda(), budget,
                            recent, nk, nv, perm.cuda(), stream=stream)
    torch.cuda.synchronize()
    return [t.cpu() for t in got] + [nk.cpu(), nv.cpu(), perm]


def check(cache, w, budget, recent, got):
    length, index, kept_w, nk, nv, perm = got
    Hkv, page = w.shape[1], cache.page
    want = ref.evict(w, cache.lens, budget, recent)
    untouched = torch.ones(nk.shape[:3], dtype=torch.bool)
    for b, n in enumerate(cache.lens):
        m = min(n, budget)
        assert int(length[b]) == m
        for h in range(Hkv):
            keep = want[b, h]
            assert index[b, h].tolist() == keep + [-1] * (budget - m), (b, h)
            x = w[b, h, keep]
            assert torch.equal(kept_w[b, h, :m].view(torch.int32), x.view(torch.int32))
            assert bool((kept_w[b, h, m:] == 0).all())
            for which, new in ((0, nk), (1, nv)):
                old = cache.view(which)
                for j, s in enumerate(keep):
                    p = int(perm[b, j // page])
                    assert torch.equal(new[p, j % page, h],
                                       old[cache.table[b, s // page], s % page, h]), (b, h, j)
                    untouched[p, j % page, h] = False
    return untouched


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special"])
@pytest.mark.parametrize("D,Hkv,page,order,budget,recent", [
    (64, 1, 8, "token", 40, 0), (128, 3, 16, "head", 64, 20), (256, 2, 64, "token", 33, 33),
    (128, 2, 128, "head", 1, 0), (64, 2, 16, "token", 1, 1), (128, 1, 32, "token", 299, 100),
])
def test_against_a_sort(kind, D, Hkv, page, order, budget, recent):
    lens = [0, 1, 20, budget, budget + 1, 300]
    cache = ref.Cache(lens, page, Hkv, D, torch.bfloat16, order=order, fill=5.0, seed=budget)
    w = weights_of(len(lens), Hkv, 310, kind, seed=D)
    got = run(cache, w, budget, recent, order=order)
    untouched = check(cache, w, budget, recent, got)
    assert bool((got[3][untouched] == 7).all()) and bool((got[4][untouched] == 7).all())


def test_long_rows_of_close_weights():
    """Keys that differ in their last bits only, over many tiles of the select."""
    cache = ref.Cache([9000, 5001], 512, 1, 64, torch.float16, fill=1.0, seed=1)
    g = torch.Generator().manual_seed(2)
    bits = 0x3f800000 + torch.randint(0, 4000, (2, 1, 9000), generator=g)
    w = bits.int().view(torch.float32)
    check(cache, w, 3001, 64, run(cache, w, 3001, 64))


def test_same_pool_and_another_stream():
    cache = ref.Cache([200, 90], 16, 2, 64, torch.float16, fill=5.0, seed=3)
    w = weights_of(2, 2, 208, "random")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(cache, w, 50, 10, same_pool=True, stream=st)
    check(cache, w, 50, 10, got)
    old = cache.pools[0].shape[0]
    assert torch.equal(got[3][:old], cache.view(0)) and torch.equal(got[4][:old], cache.view(1))


def test_bad_requests_copy_nothing():
    cache = ref.Cache([100, 100, 100, 100, 30], 16, 1, 64, torch.bfloat16, fill=5.0, seed=4)
    w = weights_of(5, 1, 112, "random")
    k, v = cache.view(0, "cuda"), cache.view(1, "cuda")
    nk, nv = torch.full((15, 16, 1, 64), 7.0, dtype=k.dtype, device="cuda"), None
    nv = nk.clone()
    new = torch.arange(15).view(5, 3).int()
    table, lens = cache.table.clone(), cache.seq_len.clone()
    lens[0], lens[1] = -1, 113
    table[2, 6] = k.shape[0]
    new[3, 2] = 15
    got = sv.kv_cache_evict(k, v, table.cuda(), lens.cuda(), w.cuda(), 40, 8, nk, nv, new.cuda())
    length, index, kept = (t.cpu() for t in got)
    assert length.tolist() == [-1, -1, -1, -1, 30]
    assert bool((index[:4] == -1).all()) and bool((kept[:4] == 0).all())
    assert index[4, 0].tolist() == list(range(30)) + [-1] * 10
    assert bool((nk[:12] == 7).all()) and bool((nv[:12] == 7).all())
    assert torch.equal(nk[12].cpu(), cache.view(0)[table[4, 0]])


def test_an_evicted_cache_attends_as_its_kept_keys():
    """Eviction that drops only keys of no weight leaves the attention as it was."""
    cache = ref.Cache([150], 16, 1, 128, torch.bfloat16, seed=5)
    q = torch.randn((1, 1, 4, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    got = run(cache, weights_of(1, 1, 150, "random"), 60, 20)
    length, index, _, nk, nv, perm = got
    out, _ = sv.paged_attention(q.cuda(), nk.cuda(), nv.cuda(), perm.cuda(), length.cuda())
    keep = index[0, 0].long()
    k, v = cache.row(0, 0, 0)[keep], cache.row(1, 0, 0)[keep]
    for h in range(4):
        p = torch.softmax(k @ q[0, 0, h].double() / 128 ** 0.5, 0)
        assert ref.close(out[0, 0, h].cpu(), p @ v, (p @ v.abs()) * 2.0 ** -7)
