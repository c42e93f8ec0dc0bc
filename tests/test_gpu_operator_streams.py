"""The calls around the verify on a stream that is not torch's current one, with outputs they make
themselves: what the current stream still has to do reaches none of them."""
import pytest
import torch

import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu

BUSY = 200_000_000  # clocks the current stream is held for (0.1 s)


def inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    d = dict(q=rand(4, 3, 8, 64).bfloat16(), k=rand(64, 16, 2, 64).bfloat16(),
             v=rand(64, 16, 2, 64).bfloat16(),
             table=torch.arange(64, device="cuda").int().view(4, 16),
             lens=torch.tensor([200, 3, 256, 77], device="cuda").int(),
             logits=rand(4, 3, 1000), presence=torch.full((4,), 0.5, device="cuda"), new_k=torch.zeros(16, 16, 2, 64, device="cuda").bfloat16(),
             new_table=torch.arange(16, device="cuda").int().view(4, 4))
    d["new_v"] = d["new_k"].clone()
    d["lse"] = sv.paged_attention(d["q"], d["k"], d["v"], d["table"], d["lens"])[1]
    d["weights"] = sv.attention_weight_sum(d["q"], d["k"], d["table"], d["lens"], d["lse"])
    return d


CALLS = {
    "adjust": lambda d, **kw: (sv.logit_adjust(d["logits"], presence=d["presence"], **kw),),
    "attend": lambda d, **kw: sv.paged_attention(
        d["q"], d["k"], d["v"], d["table"], d["lens"], **kw),
    "weigh": lambda d, **kw: (sv.attention_weight_sum(
        d["q"], d["k"], d["table"], d["lens"], d["lse"], **kw),),
    "evict": lambda d, **kw: sv.kv_cache_evict(
        d["k"], d["v"], d["table"], d["lens"], d["weights"], 50, 10, d["new_k"], d["new_v"],
        d["new_table"], **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_made_by_the_call_belong_to_its_stream(name):
    d, call, st = inputs(), CALLS[name], torch.cuda.Stream()
    want = [t.clone() for t in call(d)]
    call(d, stream=st)  # (anything made once is made here)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the outputs' sizes that the current stream frees, and writes to later
    freed = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(BUSY)
    for t in freed:
        t.fill_(77)
    del freed, t
    got = call(d, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_default_key_weights_are_cleared_on_the_calls_stream():
    d, st = inputs(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)  # a clear on the current stream would come after this
    got = CALLS["weigh"](d, stream=st)[0]
    with torch.cuda.stream(st):
        soon = got.clone()
    torch.cuda.synchronize()
    assert torch.equal(soon, d["weights"]) and torch.equal(got, d["weights"])
