"""Workspaces of calls that are captured into CUDA graphs: a graph's own, shared with nothing."""
import pytest
import torch

import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def attend(B, P, G, D, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    cols = -(-n // 64)
    k, v, q = rand(B * cols, 64, 2, D), rand(B * cols, 64, 2, D), rand(B, P, 2 * G, D)
    table = torch.arange(B * cols, device="cuda").int().view(B, cols)
    lens = torch.full((B,), n, device="cuda").int()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    return lambda **kw: sv.paged_attention(q, k, v, table, lens, out=out, out_lse=lse, **kw)


def verify(B, k, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((B, k + 1, V), generator=g, device="cuda")
    d = torch.randn((B, k, V), generator=g, device="cuda")
    x = torch.randint(0, V, (B, k), generator=g, device="cuda").int()
    u = torch.rand((B, k + 1), generator=g, device="cuda")
    outs = (torch.zeros((B, k + 1), device="cuda").int(), torch.zeros(B, device="cuda").int())
    return lambda **kw: sv.spec_verify_sample(z, d, x, u, 0.8, out_tokens=outs[0],
                                              out_accept_len=outs[1], want_probs=False, **kw)[:2]


@pytest.mark.parametrize("make", [lambda s: attend(8, 3, 4, 128, 3000 + s, s),
                                  lambda s: verify(8, 3, 30000, s)], ids=["attend", "verify"])
@pytest.mark.parametrize("given", [False, True])
def test_graphs_have_workspaces_of_their_own(make, given):
    calls = [make(s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in calls]
    want = [[t.clone() for t in call()] for call in calls]
    torch.cuda.synchronize()
    kept = {key: ws.data_ptr() for key, ws in sv._ws_cache.items()}
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side if given else None):
            outs.append(call(stream=side) if given else call())
    # nothing that was kept for eager calls is in a graph, and nothing of a graph is kept
    assert {key: ws.data_ptr() for key, ws in sv._ws_cache.items()} == kept
    torch.cuda.synchronize()
    for _ in range(20):
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_a_graph_outlives_a_larger_eager_call():
    small, large = attend(2, 1, 4, 64, 3000, 3), attend(2, 9, 7, 128, 3000, 4)
    want = [t.clone() for t in small()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = small()
    large()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # what the allocator has to give now is not what the graph writes to
    others = [torch.full((1 << 20,), 5, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(bool((t == 5).all()) for t in others)
