"""The bounded waits of logit_adjust, driven to their limit: the call ends on its own, and the rows whose
copies it gave up on are NaN as a whole."""
import pytest
import torch

import speculative_decoding_verification_17_gb300 as sv

INVALID = 1


def test_the_limit_is_checked():
    for us in (0, 999, 100001):
        assert sv.library().logit_adjust_wait_selftest(
            None, 0, 0, 0, *[None] * 3, 0, *[None] * 7, 0, None, 1, 1, 8, None, 0, 0, us, None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,P,V", [(24, 6, 32768), (3, 9, 2048), (2, 3, 4104), (2, 1, 8192), (2, 5, 4099)])
def test_rows_that_were_given_up_are_nan(dtype, B, P, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((B, P, V), generator=g, device="cuda").to(dtype)
    history = torch.randint(0, V, (B, 300), generator=g, device="cuda").int()
    n = torch.full((B,), 300, device="cuda").int()
    nd = torch.randint(0, P, (B,), generator=g, device="cuda").int()
    nd[0] = P - 1
    pi = torch.full((B,), 0.5, device="cuda")
    want, out = torch.full_like(z, 7.0), torch.full_like(z, 7.0)
    sv.logit_adjust(z, history, n, presence=pi, num_draft=nd, out=want)
    code = sv.SV_F32 if dtype == torch.float32 else sv.SV_BF16
    assert sv.library().logit_adjust_wait_selftest(
        z.data_ptr(), P * V, V, code, history.data_ptr(), n.data_ptr(), None, 300, None,
        nd.data_ptr(), None, pi.data_ptr(), None, None, None, 0, None, B, P, V, out.data_ptr(), P * V,
        V, 1000, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    pieces = V % 8 == 0  # else element by element, without waits
    rows = torch.arange(P, device="cuda")
    gone = ((rows >= 2) & (rows <= nd[:, None])) if pieces else torch.zeros((B, P), device="cuda").bool()
    assert bool(out[gone].isnan().all()) and torch.equal(out[~gone], want[~gone])
    sv.logit_adjust(z, history, n, presence=pi, num_draft=nd, out=out)
    assert torch.equal(out, want)
