"""qk_norm_rotate of heads near the ends of their type's range, whose squares fp32 does not hold."""
import math

import pytest
import torch

import kv8_reference as ref8
import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30, 1e-6])
@pytest.mark.parametrize("D,R,interleaved", [(64, 64, False), (128, 32, True), (256, 256, False)])
def test_heads_near_the_ends_of_their_range(D, R, interleaved, eps):
    """Squares of bf16 heads that pass fp32's range, above or below."""
    sizes = [-130, -120, -100, -76, -70, -64, -52, -48, -40, 0, 40, 57, 60, 63, 64, 90, 120, 125]
    g = torch.Generator().manual_seed(D)
    x = torch.randn((len(sizes), 3, D), generator=g, dtype=torch.float64).clamp(-3.9, 3.9)
    x = (x * torch.exp2(torch.tensor(sizes, dtype=torch.float64))[:, None, None]).to(torch.bfloat16)
    x[::2, 1, ::2] = 0.0
    x[13, 2, 5], x[15, 2, 3] = 2.0 ** -60, 1.0  # small beside what is large
    pos = torch.arange(len(sizes)).int()
    freq = 10000.0 ** (-torch.arange(R // 2) * 2.0 / R)
    w = 1 + 0.3 * torch.randn(D, generator=g)
    for weight in (w, None):
        wd = None if weight is None else weight.cuda()
        out, _ = sv.qk_norm_rotate(x.cuda(), x[:, :1].contiguous().cuda(), pos.cuda(), freq.cuda(), q_weight=wd,
                                   eps=eps, interleaved=interleaved)
        want, tol = ref8.norm_rotate(x, pos, freq, weight, float(torch.tensor(eps)), True, interleaved)
        assert ref.close(out.cpu(), want, tol)


def test_heads_of_zeros_and_infinities_keep_their_results():
    q = torch.zeros((5, 2, 128), dtype=torch.bfloat16)
    q[1, 0, 7], q[2, 1, 3] = math.inf, -math.inf
    q[3] = 2.0 ** 120
    q[4, 1] = 2.0 ** -120
    for eps in (0.0, 1e-6):
        out, _ = sv.qk_norm_rotate(q.cuda(), q.cuda(), torch.zeros(5).int().cuda(), eps=eps)
        out = out.cpu()
        zero = out[0].isnan().all() if eps == 0 else (out[0] == 0).all()
        assert bool(zero) and bool(out[1, 0, 7].isnan()) and bool((out[1, 0, 8:] == 0).all())
        assert bool(out[2, 1, 3].isnan()) and bool((out[3] == 1).all())
        assert bool((out[4, 1] == (1 if eps == 0 else 0)).all()) or eps > 0


@pytest.mark.parametrize("D,heads,T", [(64, 21, 1300), (128, 11, 1300), (256, 5, 1300), (128, 70, 7)])
def test_heads_out_of_range_among_others_and_in_place(D, heads, T):
    """A warp per row and a CTA per row, several turns of heads; results that go where the rows lay are
    those of a call into other memory."""
    g = torch.Generator().manual_seed(heads)
    sizes = torch.tensor([-120.0, -60.0, 0.0, 0.0, 0.0, 62.0, 110.0])[torch.randint(0, 7, (T, heads), generator=g)]
    x = (torch.randn((T, heads, D), generator=g).clamp(-3.9, 3.9) * torch.exp2(sizes)[..., None]).to(torch.bfloat16)
    pos, freq = torch.arange(T).int(), 10000.0 ** (-torch.arange(D // 2) * 2.0 / D)
    weight = torch.where(torch.arange(D) % 5 == 0, 0.0, 2.0)
    k = torch.zeros((T, 1, D), dtype=torch.bfloat16, device="cuda")
    args = (pos.cuda(), freq.cuda())
    kw = dict(q_weight=weight.cuda(), k_weight=weight.cuda(), eps=0.0)
    out, _ = sv.qk_norm_rotate(x.cuda(), k, *args, **kw)
    want, tol = ref8.norm_rotate(x, pos, freq, weight, 0.0, True, False)
    assert ref.close(out.cpu(), want, tol)
    here = x.cuda()
    sv.qk_norm_rotate(here, k, *args, **kw, out_q=here)
    assert torch.equal(here, out)
