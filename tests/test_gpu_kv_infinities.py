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
