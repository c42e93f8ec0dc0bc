"""How exactly paged_attention holds its weights: far below the output's rounding, and small ones too."""
import pytest
import torch

import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,G,P,n", [(64, 4, 1, 200), (128, 4, 1, 1000), (128, 4, 6, 300),
                                     (64, 8, 8, 500), (128, 8, 9, 200), (256, 4, 3, 400),
                                     (256, 8, 8, 300)])
def test_weights_keep_more_bits_than_their_type(dtype, D, G, P, n):
    """Nearly equal weights of values of both signs: outputs far smaller than what they sum."""
    cache = ref.Cache([n, n - 3], 64, 1, D, dtype, seed=D + n)
    q = (torch.randn((2, P, G, D), generator=torch.Generator().manual_seed(n)) * 0.05).to(dtype)
    nd = [P - 1, 0]
    out, _ = sv.paged_attention(q.cuda(), cache.view(0, "cuda"), cache.view(1, "cuda"),
                                cache.table.cuda(), cache.seq_len.cuda(),
                                num_draft=torch.tensor(nd).int().cuda())
    out = out.cpu()
    half = ref.HALF_STEP[dtype]
    two_halves = half ** 2  # of a weight: what is left after its high and its low half
    for b in range(2):
        k, v = cache.row(0, b, 0), cache.row(1, b, 0)
        for i in range(nd[b] + 1):
            pos = cache.lens[b] - 1 - nd[b] + i
            for head in range(G):
                s, sees, err = ref.score_row(q[b, i, head].double(), k, pos, scale=D ** -0.5)
                p = torch.softmax(s[sees], 0)
                o, size = p @ v[sees], p @ v[sees].abs()
                # scores (in the weight and in the sum), the exponential, sums of fp32, two halves
                w = 2 * float(err[sees].max()) + 2.0 ** -21 + (n + 8) * 2.0 ** -23 + two_halves
                small = 2.0 ** -24 if dtype == torch.float16 else 1e-30
                assert ref.close(out[b, i, head], o, w * size + half * o.abs() + small), (b, i, head)


@pytest.mark.parametrize("D,G,P", [(64, 1, 1), (128, 4, 1), (128, 4, 6), (128, 8, 9), (256, 8, 4)])
@pytest.mark.parametrize("below", [25.4, 27.0, 29.7])
def test_a_long_tail_of_small_fp16_weights(D, G, P, below):
    """One key near the end whose score is far above all others: these weigh 2^-below of it each, but
    there are 16384 of them in one CTA's range. The requests share their pages."""
    n, B = 16384, 160
    k = torch.zeros((n // 128, 128, 1, D), dtype=torch.float16, device="cuda")
    v = torch.ones_like(k)
    q = torch.zeros((B, P, G, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    k[(n - P) // 128, (n - P) % 128, 0, 0] = 1.0
    v[(n - P) // 128, (n - P) % 128] = 0.0
    table = torch.arange(n // 128, device="cuda").int().expand(B, -1).contiguous()
    lens = torch.full((B,), n, device="cuda").int()
    scale = below * 0.6931471805599453
    out, lse = sv.paged_attention(q, k, v, table, lens, scale=scale)
    # row i sees n - P + 1 + i keys, all but one of them of the tail
    rows = torch.arange(P, device="cuda").double() + n - P
    tail = rows * torch.exp(-torch.tensor(scale, dtype=torch.float64))
    want = (tail / (1 + tail))[None, :, None, None].expand(B, P, G, D)
    # each weight is 2^(7 - below), on fp16's grid of 2^-24 after the lift: off by 2^-25 at most; a
    # score of ~20 in fp32 and its scaling: 2^-18; the sums; the output's rounding and subnormals
    tol = want * (2.0 ** (below - 32) + 2.0 ** -16 + n * 2.0 ** -23 + 2.0 ** -11) + 2.0 ** -24
    assert ref.close(out, want, tol)
    assert torch.allclose(lse.double(), (scale + torch.log1p(tail))[None, :, None].expand(B, P, G),
                          rtol=0, atol=2.0 ** -16)


@pytest.mark.parametrize("D,G,P", [(64, 1, 1), (64, 8, 4), (128, 4, 1), (128, 4, 6), (128, 16, 2),
                                   (256, 2, 5), (256, 8, 3)])
def test_bf16_weights_keep_the_bits_of_fp32(D, G, P):
    """Up to 32 rows per kv head. Three keys: weights 1, 1 and p, values -c1, -c2 and 1, where c1 and c2
    are the first 16 bits of p: what is left is p's third part."""
    x = torch.arange(0xbc00, 0xbf80).to(torch.int16).view(torch.bfloat16)  # all in (-1, -2^-7]
    p = torch.exp(x.double())
    c1 = p.bfloat16()
    c2 = (p - c1.double()).bfloat16()
    # the scores whose weight has the largest third parts, up to 2^-18
    some = (p - c1.double() - c2.double()).abs().topk(96).indices
    x, p, c1, c2, B = x[some], p[some], c1[some], c2[some], 96
    n, page = 2 + P, 8 if P <= 6 else 16  # the drafts' own keys come last: of no weight to anything
    k = torch.zeros((B, page, 1, D), dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    k[:, 2, 0, 0] = x
    k[:, 3:, 0, 0] = -1000.0
    v[:, 0, 0], v[:, 1, 0], v[:, 2, 0] = -c1[:, None], -c2[:, None], 1.0
    q = torch.zeros((B, P, G, D), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    table = torch.arange(B).int()[:, None]
    lens = torch.full((B,), n).int()
    out, _ = sv.paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda(), scale=1.0)
    want = ((p - c1.double() - c2.double()) / (2 + p))[:, None, None, None].expand(B, P, G, D)
    # the exponential and its argument 2^-21, the three parts 2^-24, sums of numbers near 1 in fp32
    # 2^-22; the output's rounding
    tol = ((2.0 ** -21 + 2.0 ** -24 + 2.0 ** -22) / (2 + p))[:, None, None, None] + 2.0 ** -8 * want.abs()
    assert bool((want.abs() > 2 * tol).all())  # (two parts would leave it out)
    assert ref.close(out.cpu(), want, tol)
