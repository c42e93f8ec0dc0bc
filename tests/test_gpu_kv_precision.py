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
