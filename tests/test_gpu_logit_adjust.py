"""logit_adjust against its definition in 64 bits, where it can go wrong: vocabularies no vector
divides, chunk borders, rows that lie apart, masks that leave a row empty, NaN and infinities
under the mask, drafts that repeat, duplicate biases, and requests with bad counts."""
import math

import pytest
import torch

import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def case(B, P, V, dtype, *, H=50, bias=0, mask=None, seed=0, prompt=True, zipf=True):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    tok = lambda *s: (V ** rand(*s) - 1 if zipf else V * rand(*s)).long().clamp(0, V - 1).int()  # noqa: E731
    d = dict(logits=(torch.randn((B, P, V), generator=g) * 3).to(dtype))
    if H:
        d["history"] = tok(B, H)
        d["hist_len"] = torch.randint(0, H + 1, (B,), generator=g).int()
        if prompt:
            d["prompt_len"] = (d["hist_len"] * rand(B)).int()
    if P > 1:
        d["draft"] = tok(B, P - 1)
        d["num_draft"] = torch.randint(0, P, (B,), generator=g).int()
    d["repetition"], d["presence"], d["frequency"] = 1 + rand(B), rand(B) - 0.3, rand(B)
    if bias:
        d["bias_tokens"] = torch.randint(-2, V + 2, (B, bias), generator=g).int()
        d["bias_values"] = 20 * rand(B, bias) - 10
    if mask is not None:
        words = torch.randint(-2 ** 31, 2 ** 31, (B, P, -(-V // 32)), generator=g)
        d["allowed"] = {"half": words, "none": words * 0, "all": words * 0 - 1}[mask].int()
    return d


def call(d, dev="cuda", **kw):
    t = {k: v.to(dev) for k, v in d.items()}
    out = kw.pop("out", None)
    if out is None:
        out = torch.full_like(t["logits"], 7.0)
    got = sv.logit_adjust(t["logits"], t.get("history"), t.get("hist_len"),
                          prompt_len=t.get("prompt_len"), draft_tokens=t.get("draft"),
                          num_draft=t.get("num_draft"), repetition=t.get("repetition"),
                          presence=t.get("presence"), frequency=t.get("frequency"),
                          bias_tokens=t.get("bias_tokens"), bias_values=t.get("bias_values"),
                          allowed=t.get("allowed"), out=out, **kw)
    torch.cuda.synchronize()
    return got.cpu()


def check(d, got, before=7.0):
    want, tol = ref.adjust(**d)
    live = ~tol[:, :, 0].isnan()
    assert ref.close(got[live], want[live], tol[live])
    if before is not None:
        assert bool((got[~live] == before).all()), "a row past num_draft was written"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,P,V,H,bias,mask", [
    (1, 1, 1, 3, 0, None), (1, 2, 7, 20, 4, "half"), (2, 3, 33, 64, 5, "half"),
    (3, 5, 1000, 700, 0, "half"), (2, 9, 8192, 300, 40, None), (2, 2, 8193, 300, 70, "half"),
    (2, 17, 4104, 2500, 300, "half"), (1, 4, 50257, 900, 3, "all"), (5, 3, 2048, 0, 0, "none"),
    (2, 2, 32000, 0, 9, None), (1, 1, 20000, 1, 0, None),
])
def test_against_definition(dtype, B, P, V, H, bias, mask):
    d = case(B, P, V, dtype, H=H, bias=bias, mask=mask, seed=V + P, prompt=P % 2 == 1)
    check(d, call(d))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [1500, 2047, 5000])
@pytest.mark.parametrize("V", [4104, 12296, 33000])
def test_long_histories(dtype, H, V):
    # (more than a thread's batch of loads, in fours and one by one; a short last chunk)
    d = case(3, 4, V, dtype, H=H, bias=30, mask="half", seed=V + H, zipf=H != 5000)
    d["hist_len"][0] = H
    got = call(d)
    check(d, got)
    d["hist_len"][1] = H + 1  # refused; the others are as they were
    again = call(d)
    assert bool(again[1, :d["num_draft"][1] + 1].isnan().all())
    assert torch.equal(again[0], got[0]) and torch.equal(again[2], got[2])


def test_every_option_alone():
    full = case(3, 4, 640, torch.float32, H=200, bias=20, mask="half", seed=5)
    for keep in (("history", "hist_len"), ("draft",), ("bias_tokens", "bias_values"),
                 ("allowed",), (), ("num_draft",)):
        for rule in ((), ("repetition",), ("presence",), ("frequency",)):
            d = {k: v for k, v in full.items() if k in ("logits",) + keep + rule}
            check(d, call(d))


def test_masked_values_do_not_matter_and_empty_rows():
    d = case(2, 3, 1024, torch.bfloat16, H=100, mask="half", seed=2)
    d["num_draft"][:] = 2
    d["allowed"][0, 1] = 0
    bits = ((d["allowed"][..., None] >> torch.arange(32).int()) & 1).bool().flatten(2)
    junk = torch.tensor([math.nan, math.inf, -math.inf])[torch.randint(0, 3, bits.shape)]
    d["logits"] = torch.where(bits, d["logits"].float(), junk).to(torch.bfloat16)
    got = call(d)
    check(d, got)
    assert bool((got[~bits] == -math.inf).all()) and bool((got[0, 1] == -math.inf).all())


def test_unmasked_nan_and_infinities_pass_through():
    d = case(1, 1, 64, torch.float32, H=30, seed=3)
    d["logits"][0, 0, :6] = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 3e38])
    d["history"][0, :3] = torch.tensor([0, 1, 2])
    d["hist_len"][0] = 30
    check(d, call(d))


def test_repeated_drafts_and_duplicate_biases():
    d = case(2, 6, 96, torch.float32, H=0, bias=40, seed=4)
    d["draft"] = torch.tensor([[5, 5, 9, 5, 9], [0, 95, 95, -1, 200]]).int()
    d["num_draft"] = torch.tensor([5, 5]).int()
    d["bias_tokens"] = (d["bias_tokens"] % 12).int()
    check(d, call(d))


def test_one_token_repeated_and_every_token_seen():
    d = case(2, 2, 256, torch.float32, H=20000, seed=6, zipf=False)
    d["history"][0] = 17
    d["hist_len"][:] = 20000
    check(d, call(d))


@pytest.mark.parametrize("pad", [8, 3])
def test_rows_apart_in_place_and_another_stream(pad):
    d = case(3, 3, 520, torch.bfloat16, H=60, mask="half", seed=7)
    wide = torch.full((3, 4, 520 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    view = wide[:, :3, :520]
    view.copy_(d["logits"])
    t = {k: v.cuda() for k, v in d.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    args = dict(prompt_len=t["prompt_len"], draft_tokens=t["draft"], num_draft=t["num_draft"],
                repetition=t["repetition"], presence=t["presence"], frequency=t["frequency"],
                allowed=t["allowed"])
    flat = torch.zeros((3, 3, 520), dtype=torch.bfloat16, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    sv.logit_adjust(view, t["history"], t["hist_len"], out=flat, stream=st, **args)
    sv.logit_adjust(view, t["history"], t["hist_len"], out=view, stream=st, **args)
    torch.cuda.synchronize()
    check(d, flat.cpu(), before=0.0)
    check(d, view.cpu(), before=None)
    assert bool((wide[:, 3] == 7).all()) and bool((wide[:, :, 520:] == 7).all())


def test_bad_counts_give_nan():
    for name, value in (("hist_len", -1), ("hist_len", 51), ("prompt_len", -1),
                        ("prompt_len", 51), ("num_draft", -1), ("num_draft", 3)):
        d = case(3, 3, 300, torch.float32, H=50, seed=8)
        d[name][1] = value
        got = call(d)
        assert bool(got[1].isnan().all())
        ok = {k: v[[0, 2]] for k, v in d.items()}
        check(ok, got[[0, 2]])


def test_graph_replay_and_no_requests():
    d = case(2, 3, 5000, torch.bfloat16, H=100, bias=3, mask="half", seed=9)
    want = call(d)
    t = {k: v.cuda() for k, v in d.items()}
    out = torch.full_like(t["logits"], 7.0)
    run = lambda: sv.logit_adjust(  # noqa: E731
        t["logits"], t["history"], t["hist_len"], prompt_len=t["prompt_len"],
        draft_tokens=t["draft"], num_draft=t["num_draft"], repetition=t["repetition"],
        presence=t["presence"], frequency=t["frequency"], bias_tokens=t["bias_tokens"],
        bias_values=t["bias_values"], allowed=t["allowed"], out=out)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    assert sv.logit_adjust(t["logits"][:0]).shape == (0, 3, 5000)


def test_feeds_the_verify():
    """Adjusted rows go into the verify: a token the mask forbids is never emitted."""
    d = case(4, 4, 3000, torch.float32, H=80, mask="half", seed=10)
    d["num_draft"][:] = 3
    out = call(d).cuda()
    draft_logits = torch.zeros((4, 3, 3000), device="cuda")
    tokens, n, *_ = sv.spec_verify_sample(out, draft_logits, d["draft"].cuda(),
                                          torch.rand((4, 4), device="cuda"), 1.0)
    for b in range(4):
        for i, t in enumerate(tokens[b, :n[b] + 1].tolist()):
            assert (int(d["allowed"][b, i, t // 32]) >> (t % 32)) & 1
