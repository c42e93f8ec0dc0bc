"""The C ABI from several host threads at once: calls of different sizes of one kernel."""
import threading

import pytest
import torch

import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logit_adjust_of_two_sizes(dtype):
    L, code = sv.library(), sv.SV_F32 if dtype == torch.float32 else sv.SV_BF16
    jobs, errors = [], []
    for B, V in ((1, 4096), (64, 32000)):  # the smallest chunks, and the largest
        z = torch.randn((B, 2, V), device="cuda").to(dtype)
        pi = torch.full((B,), 0.5, device="cuda")
        history = torch.randint(0, V, (B, 64), device="cuda").int()
        n = torch.full((B,), 64, device="cuda").int()
        jobs.append((z, pi, history, n, torch.empty_like(z), torch.cuda.Stream()))
    want = [sv.logit_adjust(z, h, n, presence=pi) for z, pi, h, n, _, _ in jobs]
    torch.cuda.synchronize()
    go = threading.Barrier(len(jobs))

    def work(z, pi, history, n, out, st):
        B, P, V = z.shape
        args = (z.data_ptr(), P * V, V, code, history.data_ptr(), n.data_ptr(), None, 64, None, None,
                None, pi.data_ptr(), None, None, None, 0, None, B, P, V, out.data_ptr(), P * V, V,
                st.cuda_stream)
        go.wait()
        for _ in range(3000):
            if (status := L.logit_adjust(*args)) != 0:
                errors.append((tuple(z.shape), status))
                return

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for j, w in zip(jobs, want):
        assert torch.equal(j[4], w)
