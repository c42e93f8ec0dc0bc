"""Infinite keys and values that rows see: an infinitely low score is a weight of 0, and what the
definition in 64 bits makes infinite comes out infinite, wherever the key lies."""
import math

import pytest
import torch

import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("G,P", [(1, 1), (4, 1), (3, 5), (8, 5), (7, 9)])
def test_keys_of_infinitely_low_scores_weigh_nothing(G, P, dtype):
    D, lens = 64, [400, 140, 1, 257]
    cache = ref.Cache(lens, 16, 2, D, dtype, seed=1)
    g = torch.Generator().manual_seed(2)
    q = torch.randn((4, P, 2 * G, D), generator=g).to(dtype)
    q[..., 3] = q[..., 3].abs() + 0.5
    low = [(0, 5), (0, 130), (0, 131), (0, 260), (0, 390), (1, 0), (1, 139), (3, 255), (3, 256)]
    view = cache.view(0)
    for b, j in low:
        view[cache.table[b, j // 16], j % 16, :, 3] = -math.inf
    nd = [min(P - 1, x) for x in (P - 1, 2, 0, 1)]
    dev = [t.cuda() for t in (q, cache.view(0), cache.view(1), cache.table, cache.seq_len)]
    num = torch.tensor(nd).int().cuda()
    out, lse = sv.paged_attention(*dev, num_draft=num)
    prior = torch.rand((4, 2, 400), generator=g)
    w = sv.attention_weight_sum(dev[0], dev[1], dev[3], dev[4], lse, num_draft=num,
                                prior=prior.cuda(), out=torch.full((4, 2, 400), 7.0).cuda()).cpu()
    # the reference with a key of zeros there, which it then masks: the same sums of the others
    kept = [[j for j in range(n) if (b, j) not in low] for b, n in enumerate(lens)]
    for b, n in enumerate(lens):
        for h in range(2):
            k, v = cache.row(0, b, h)[kept[b]], cache.row(1, b, h)[kept[b]]
            pos_of = torch.tensor(kept[b])
            want, size = prior[b, h, :n].double().clone(), torch.zeros(n, dtype=torch.float64)
            for i in range(nd[b] + 1):
                pos = n - 1 - nd[b] + i
                sees = pos_of <= pos
                for head in range(h * G, (h + 1) * G):
                    got = out[b, i, head].cpu()
                    if not bool(sees.any()):
                        assert bool((got == 0).all()) and lse[b, i, head] == -math.inf
                        continue
                    s = (k @ q[b, i, head].double() / D ** 0.5)[sees]
                    p = torch.softmax(s, 0)
                    o = p @ v[sees]
                    # (weights rounded once to the type, the output once)
                    tol = 3 * ref.HALF_STEP[dtype] * (p @ v[sees].abs()) + 2.0 ** -20
                    assert ref.close(got, o, tol), (b, i, head)
                    assert abs(float(lse[b, i, head]) - float(torch.logsumexp(s, 0))) < 1e-4
                    want[pos_of[sees]] += p
                    size[pos_of[sees]] += p
            # scores of 64 products in fp32, exponentials and sums: far below 2^-14 of the weights
            assert ref.close(w[b, h, :n], want, 2.0 ** -14 * size + 2.0 ** -22), (b, h)
            assert bool((w[b, h, n:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,G,P,page,window", [
    (64, 1, 1, 16, 0), (128, 4, 1, 64, 0), (128, 3, 5, 16, 0), (128, 8, 6, 32, 300),
    (64, 16, 8, 128, 0), (256, 4, 3, 16, 0), (256, 8, 8, 64, 4), (128, 2, 3, 8, 2),
])
def test_values_that_are_not_finite(dtype, D, G, P, page, window):
    """Infinite and NaN values of keys anywhere (full tiles, the last, a window's first): every row's
    component is the sum of those it sees, and no other component or row is touched."""
    Hkv, lens = 2, [3000, 700, 129, 128, 2]
    B = len(lens)
    nd = [P - 1, 0, P - 1, min(1, P - 1), 0]
    g = torch.Generator().manual_seed(D + P)
    cols = -(-max(lens) // page)
    counts = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(counts), generator=g).int()
    table, at = torch.full((B, cols), -1).int(), 0
    for b, c in enumerate(counts):
        table[b, :c] = ids[at:at + c]
        at += c
    k, v = (torch.randn((sum(counts), page, Hkv, D), generator=g).to(dtype) for _ in range(2))
    q = torch.randn((B, P, Hkv * G, D), generator=g).to(dtype)
    put = lambda b, j, h, d, x: v[int(table[b, j // page]), j % page, h].__setitem__(d, x)  # noqa: E731
    inf = math.inf
    for b, n in enumerate(lens):
        first = max(0, n - 1 - nd[b] - window + 1) if window else 0
        for d, j in enumerate([first, first + 1, (first + n) // 2, n - 1, n - 2, 5, 127, 128]):
            if 0 <= j < n:
                put(b, j, 0, d, -inf if d % 2 else inf)
                put(b, j, 1, d + 8, math.nan if d == 2 else inf)
        for j, x in ((n // 3, inf), (n - 1, -inf), ((first + n) // 2, inf)):  # several of one component
            put(b, j, 1, 30, x)
    args = [t.cuda() for t in (q, k, v, table, torch.tensor(lens).int())]
    num = torch.tensor(nd).int().cuda()
    out, lse = sv.paged_attention(*args, num_draft=num, window=window)
    clean = torch.where(v.isfinite(), v, torch.zeros((), dtype=dtype))
    fine, lse_fine = sv.paged_attention(args[0], args[1], clean.cuda(), *args[3:], num_draft=num,
                                        window=window)
    out, lse, fine, lse_fine = (t.cpu() for t in (out, lse, fine, lse_fine))
    for b, n in enumerate(lens):
        j = torch.arange(n)
        rows = v[table[b, :counts[b]].long()].flatten(0, 1)[:n].double()  # [n, Hkv, D]
        odd = torch.where(rows.isfinite(), 0.0, rows)
        for i in range(nd[b] + 1):
            pos = n - 1 - nd[b] + i
            sees = (j <= pos) & ((j > pos - window) if window else True)
            total = odd[sees].sum(0).repeat_interleave(G, 0)  # [Hq, D]
            got, want = out[b, i], torch.where(total.isfinite(), fine[b, i].double(), total)
            assert bool(((got.double() == want) | (got.isnan() & want.isnan())).all()), (b, i)
            assert torch.equal(lse[b, i], lse_fine[b, i])


def test_a_query_that_is_not_a_number_beside_an_infinite_value():
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((40, 64, 1, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((1, 3, 4, 128), generator=g, device="cuda").bfloat16()
    table, n = torch.arange(40, device="cuda").int()[None], torch.tensor([2500], device="cuda").int()
    want, want_lse = sv.paged_attention(q, k, v, table, n)
    q[0, 1, 2, 7] = math.nan
    v[3, 4, 0, 9] = -math.inf
    out, lse = sv.paged_attention(q, k, v, table, n)
    hit = torch.zeros((1, 3, 4), dtype=torch.bool, device="cuda")
    hit[0, 1, 2] = True
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert bool((out[~hit][:, 9] == -math.inf).all())
    rest = torch.arange(128, device="cuda") != 9
    assert torch.equal(out[~hit][:, rest], want[~hit][:, rest])
    assert torch.equal(lse[~hit], want_lse[~hit])
