"""paged_attention and attention_weight_sum against their definitions in 64 bits, where they can
go wrong: lengths of zero and one and around the tiles' edges, ragged drafts, pages that end
inside a tile, slots past the end that hold NaN, windows over pages that are gone, bad pages and
counts, non-finite drafted values, strides, streams, graphs, and offsets past 32 bits."""
import math

import pytest
import torch

import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def queries(B, P, Hq, D, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + 99)
    return (torch.randn((B, P, Hq, D), generator=g) * size).to(dtype)


def dev_args(cache, num_draft):
    return dict(k=cache.view(0, "cuda"), v=cache.view(1, "cuda"), table=cache.table.cuda(),
                seq_len=cache.seq_len.cuda(),
                num_draft=None if num_draft is None else torch.tensor(num_draft).int().cuda())


def check_attention(cache, q, num_draft, *, slopes=None, softcap=0.0, window=0, scale=None, **kw):
    B, P, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    a = dev_args(cache, num_draft)
    out = torch.full((B, P, Hq, D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((B, P, Hq), 7.0, device="cuda")
    sl = None if slopes is None else slopes.cuda()
    sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                       num_draft=a["num_draft"], scale=scale, softcap=softcap, window=window,
                       slopes=sl, out=out, out_lse=lse, **kw)
    torch.cuda.synchronize()
    nd = num_draft if num_draft is not None else [P - 1] * B
    want = ref.attention(cache, q, nd, scale=scale, softcap=softcap, window=window, slopes=slopes)
    out, lse = out.cpu(), lse.cpu()
    for b in range(B):
        for i in range(P):
            for head in range(Hq):
                if i > nd[b]:
                    assert bool((out[b, i, head] == 7).all()) and lse[b, i, head] == 7
                    continue
                o, l, tol, tol_l = want[b, i, head]
                assert ref.close(out[b, i, head], o, tol), (b, i, head)
                assert lse[b, i, head] == l or abs(float(lse[b, i, head]) - l) <= tol_l, (b, i, head)
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,Hq,Hkv,P,page,order", [
    (64, 4, 4, 1, 16, "token"), (64, 8, 2, 3, 8, "head"), (128, 8, 2, 1, 16, "head"),
    (128, 14, 2, 4, 64, "token"), (256, 4, 2, 2, 32, "token"), (256, 2, 1, 5, 256, "head"),
    (128, 6, 1, 17, 128, "token"), (64, 32, 1, 9, 512, "head"),
])
def test_lengths_and_layouts(dtype, D, Hq, Hkv, P, page, order):
    lens = [0, 1, 2, P, 63, 64, 65, 127, 128, 129, 200, 257, 391]
    nd = [min(P - 1, b % P) for b in range(len(lens))]
    cache = ref.Cache(lens, page, Hkv, D, dtype, order=order, seed=D + P)
    check_attention(cache, queries(len(lens), P, Hq, D, dtype), nd)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rule", [
    dict(softcap=5.0), dict(window=1), dict(window=100), dict(window=130, softcap=20.0),
    dict(slopes=True), dict(slopes=True, window=64, softcap=3.0), dict(scale=0.0),
    dict(scale=-0.3),
])
def test_rules(D, rule):
    rule = dict(rule)
    if rule.get("slopes"):
        rule["slopes"] = torch.tensor([0.5, 0.0, -0.01, 0.1])
    cache = ref.Cache([5, 130, 300, 513], 16, 2, D, torch.bfloat16, seed=1)
    check_attention(cache, queries(4, 4, 4, D, torch.bfloat16, size=2.0), [3, 0, 2, 3], **rule)


def test_long_caches_are_split_and_joined():
    cache = ref.Cache([3001, 17, 5000], 64, 1, 128, torch.bfloat16, seed=2)
    check_attention(cache, queries(3, 2, 4, 128, torch.bfloat16, size=3.0), [1, 1, 0])


def test_many_rows_of_one_head():
    """More query rows per kv head than one pass holds."""
    cache = ref.Cache([150, 40], 16, 1, 64, torch.float16, seed=3)
    check_attention(cache, queries(2, 9, 48, 64, torch.float16), [8, 5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,G,P,page,rule", [
    (64, 1, 1, 16, {}), (64, 5, 5, 8, {}), (64, 8, 6, 64, dict(window=300)), (64, 8, 13, 32, {}),
    (128, 4, 1, 16, dict(softcap=20.0)), (128, 4, 6, 128, {}), (128, 8, 6, 32, {}),
    (128, 16, 8, 256, dict(slopes=True)), (256, 2, 3, 16, {}), (256, 4, 7, 64, {}),
    (256, 8, 6, 16, dict(window=129)), (256, 8, 9, 8, {}),
])
def test_many_requests_share_the_ranges(dtype, D, G, P, page, rule):
    """Every width of the kernel with far more pieces than CTAs: short and long caches, empty ones
    and ones shorter than the drafts, side by side."""
    g = torch.Generator().manual_seed(D + G + P)
    B, Hkv = 150, 2
    lens = torch.cat([torch.tensor([0, 1, P, 128, 129]),
                      torch.exp(torch.rand(B - 5, generator=g) * 7.6).int().clamp(1, 2000)]).int()
    lens = lens[torch.randperm(B, generator=g)]
    nd = torch.randint(0, P, (B,), generator=g).int()
    cols = -(-int(lens.max()) // page)
    counts = -(-lens.long() // page)
    total = int(counts.sum())
    ids, table = torch.randperm(total, generator=g).int(), torch.full((B, cols), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts.tolist()):
        table[b, :c] = ids[at:at + c]
        at += c
    dg = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((total, page, Hkv, D), generator=dg, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((B, P, Hkv * G, D), generator=dg, device="cuda").to(dtype)
    table, lens, nd = table.cuda(), lens.cuda(), nd.cuda()
    rule = dict(rule)
    if rule.get("slopes"):
        rule["slopes"] = torch.rand(Hkv * G, generator=dg, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((B, P, Hkv * G), 7.0, device="cuda")
    for _ in range(2):  # (the second call finds what the first left in the workspace)
        sv.paged_attention(q, k, v, table, lens, num_draft=nd, out=out, out_lse=lse, **rule)
    acc = nd - (torch.arange(B, device="cuda") % 2).int()
    want, want_lse, tol, tol_lse, live = ref.attention_on_device(q, k, v, table, lens, nd,
                                                                 scale=D ** -0.5, **rule)
    assert ref.close(out[live], want[live], tol[live])
    assert ref.close(lse[live], want_lse[live], tol_lse[live])
    assert bool((out[~live] == 7).all()) and bool((lse[~live] == 7).all())
    # the weights of all rows up to the accepted ones: every row that sees a key gave 1 in all
    w = sv.attention_weight_sum(q, k, table, lens, lse, num_draft=nd, accept_len=acc, **rule)
    rows = torch.arange(P, device="cuda")
    gave = ((rows <= acc[:, None]) & (lens[:, None] - 1 - nd[:, None] + rows >= 0)).sum(1) * G
    assert torch.allclose(w.double().sum(-1), gave[:, None].double().expand(B, Hkv), rtol=2e-4,
                          atol=1e-12)


def test_large_scores_keep_their_range():
    cache = ref.Cache([400, 129], 16, 1, 128, torch.float16, seed=4)
    for pool in cache.pools[:1]:
        pool.mul_(torch.linspace(0.01, 30, pool.shape[1])[None, :, None, None].to(pool.dtype))
    check_attention(cache, queries(2, 3, 2, 128, torch.float16, size=8.0), [2, 2])


def test_repeats_are_identical():
    cache = ref.Cache([2000, 777], 32, 2, 128, torch.bfloat16, seed=5)
    q = queries(2, 3, 8, 128, torch.bfloat16).cuda()
    a = dev_args(cache, [2, 2])
    runs = [sv.paged_attention(q, a["k"], a["v"], a["table"], a["seq_len"],
                               num_draft=a["num_draft"]) for _ in range(3)]
    for o, l in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(l, runs[0][1])


def test_window_over_pages_that_are_gone():
    cache = ref.Cache([300, 97], 16, 2, 64, torch.bfloat16, seed=6)
    q = queries(2, 2, 4, 64, torch.bfloat16)
    for b, n in enumerate(cache.lens):
        first = n - 2 - 50 + 1  # the first key any row sees
        for t in range(first // 16):
            page = int(cache.table[b, t])
            for pool in cache.pools:
                pool[page] = math.nan
    keep = cache.table.clone()
    check_attention(cache, q, [1, 1], window=50)  # NaN in pages no row sees
    a = dev_args(cache, [1, 1])
    gone = keep.clone()
    for b, n in enumerate(cache.lens):
        gone[b, :(n - 2 - 50 + 1) // 16] = -1
    one = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                             num_draft=a["num_draft"], window=50)[0]
    two = sv.paged_attention(q.cuda(), a["k"], a["v"], gone.cuda(), a["seq_len"],
                             num_draft=a["num_draft"], window=50)[0]
    assert torch.equal(one, two) and not bool(one.isnan().any())


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_drafts_value_does_not_reach_the_rows_ahead(value):
    cache = ref.Cache([130, 66], 16, 1, 128, torch.bfloat16, seed=7)
    q = queries(2, 4, 2, 128, torch.bfloat16)
    view = cache.view(1)
    for b, n in enumerate(cache.lens):
        j = n - 2  # the third new position: rows 0 and 1 do not see it
        view[cache.table[b, j // 16], j % 16, 0, 5] = value
    a = dev_args(cache, [3, 3])
    out, _ = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"])
    out = out.cpu()
    want = ref.attention(cache, q, [3, 3], scale=128 ** -0.5)
    for (b, i, head), (o, _, tol, _) in want.items():
        got = out[b, i, head]
        dims = torch.arange(128) != 5
        assert ref.close(got[dims], o[dims], tol[dims])
        if i < 2:
            assert bool(got.isfinite().all())
        else:
            assert not math.isfinite(float(got[5]))
            assert math.isnan(value) or float(got[5]) == value


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_a_drafts_key_does_not_reach_the_rows_ahead(value):
    cache = ref.Cache([130], 16, 1, 64, torch.bfloat16, seed=8)
    q = queries(1, 3, 2, 64, torch.bfloat16)
    cache.view(0)[cache.table[0, 129 // 16], 129 % 16, 0, 3] = value
    a = dev_args(cache, [2])
    out, lse = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"])
    assert bool(out[0, :2].isfinite().all()) and bool(lse[0, :2].isfinite().all())
    if math.isnan(value):
        assert bool(out[0, 2].isnan().all())


def test_bad_requests_are_nan_and_the_others_are_not():
    cache = ref.Cache([100, 100, 100, 100, 100], 16, 2, 64, torch.float16, seed=9)
    q = queries(5, 3, 4, 64, torch.float16)
    a = dev_args(cache, [2, 2, 2, 1, 2])
    good = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                              num_draft=a["num_draft"], out=torch.full_like(q, 7.0).cuda())[0]
    a["seq_len"][0] = cache.max_pages * 16 + 1
    a["num_draft"][1] = 3
    a["seq_len"][2] = -1
    a["table"][3, 2] = a["k"].shape[0]
    out, lse = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                                  num_draft=a["num_draft"], out=torch.full_like(q, 7.0).cuda())
    assert bool(out[:3].isnan().all()) and bool(lse[:3].isnan().all())
    assert bool(out[3, :2].isnan().all()) and bool((out[3, 2] == 7).all())
    assert torch.equal(out[4], good[4])
    a["table"][3, 2] = -7
    again, _ = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                                  num_draft=a["num_draft"])
    assert bool(again[3, :2].isnan().all()) and torch.equal(again[4], good[4])


def test_strides_streams_and_graphs():
    cache = ref.Cache([333, 60], 16, 2, 128, torch.bfloat16, seed=10)
    q = queries(2, 3, 8, 128, torch.bfloat16)
    a = dev_args(cache, [2, 1])
    want = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                              num_draft=a["num_draft"], out=torch.zeros_like(q).cuda())[0]
    # queries in a fused projection's rows, keys and values side by side in one pool
    qkv = torch.randn((2, 3, 12, 128), dtype=torch.bfloat16, device="cuda")
    qkv[:, :, :8] = q.cuda()
    both = torch.full((a["k"].shape[0], 16, 2, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    both[:, :, 0], both[:, :, 1] = a["k"], a["v"]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    run = lambda **kw: sv.paged_attention(  # noqa: E731
        qkv[:, :, :8], both[:, :, 0], both[:, :, 1], a["table"], a["seq_len"],
        num_draft=a["num_draft"], out=out, **kw)
    run(stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    none = sv.paged_attention(qkv[:0, :, :8], a["k"], a["v"], a["table"][:0], a["seq_len"][:0])
    assert none[0].shape == (0, 3, 8, 128)
    assert sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                              num_draft=a["num_draft"], want_lse=False)[1] is None


def test_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31 (and byte offsets 2^32)."""
    pages = (2 ** 31) // (16 * 2 * 128) + 64
    k = torch.empty((pages, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    cache = ref.Cache([70], 16, 2, 128, torch.bfloat16, seed=11)
    table = torch.tensor([[pages - 1, 3, pages - 5, pages - 2, 0]], dtype=torch.int32)
    for t in range(5):
        src = int(cache.table[0, t])
        k[int(table[0, t])] = cache.pools[0][src].cuda()
        v[int(table[0, t])] = cache.pools[1][src].cuda()
    q = queries(1, 2, 4, 128, torch.bfloat16)
    far = sv.paged_attention(q.cuda(), k, v, table.cuda(), cache.seq_len.cuda())
    near = sv.paged_attention(q.cuda(), cache.view(0, "cuda"), cache.view(1, "cuda"),
                              cache.table.cuda(), cache.seq_len.cuda())
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    w = [sv.attention_weight_sum(q.cuda(), kk, tt.cuda(), cache.seq_len.cuda(), far[1])
         for kk, tt in ((k, table), (cache.view(0, "cuda"), cache.table))]
    assert torch.equal(w[0], w[1])


# ------------------------------------------------------------------------------ key weights
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,Hq,Hkv,P,page,order,rule", [
    (64, 4, 4, 1, 16, "token", {}), (128, 8, 2, 4, 8, "head", {}),
    (256, 4, 1, 3, 64, "token", dict(softcap=10.0)), (128, 14, 2, 9, 128, "head", dict(window=70)),
    (64, 40, 1, 5, 32, "token", dict(slopes=True)),
])
def test_key_weights(dtype, D, Hq, Hkv, P, page, order, rule):
    lens = [0, 1, P, 64, 127, 128, 129, 300]
    B = len(lens)
    nd = [min(P - 1, b % P) for b in range(B)]
    acc = [(b * 7) % (n + 2) - 1 for b, n in enumerate(nd)]
    cache = ref.Cache(lens, page, Hkv, D, dtype, order=order, seed=D + Hq)
    q = queries(B, P, Hq, D, dtype)
    rule = dict(rule)
    slopes = torch.linspace(0, 0.2, Hq) if rule.pop("slopes", False) else None
    a = dev_args(cache, nd)
    sl = None if slopes is None else slopes.cuda()
    _, lse = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"],
                                num_draft=a["num_draft"], slopes=sl, **rule)
    g = torch.Generator().manual_seed(3)
    prior = torch.rand((B, Hkv, 310), generator=g)
    apart = lse.permute(0, 2, 1).contiguous().permute(0, 2, 1)  # lse of any strides
    got = sv.attention_weight_sum(q.cuda(), a["k"], a["table"], a["seq_len"], apart,
                                  num_draft=a["num_draft"],
                                  accept_len=torch.tensor(acc).int().cuda(), slopes=sl,
                                  prior=prior.cuda(), out=torch.full_like(prior, 7.0).cuda(),
                                  **rule).cpu()
    want, tol = ref.weight_sum(cache, q, nd, acc, lse.cpu(), prior, scale=D ** -0.5,
                               slopes=slopes, **rule)
    for b, n in enumerate(lens):
        assert ref.close(got[b, :, :n], want[b, :, :n], tol[b, :, :n]), b
        assert bool((got[b, :, n:] == 7).all())


def test_key_weights_in_place_add_up_to_the_rows():
    cache = ref.Cache([500, 90], 16, 2, 128, torch.bfloat16, seed=12)
    q = queries(2, 3, 8, 128, torch.bfloat16)
    a = dev_args(cache, None)
    _, lse = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"])
    w = torch.zeros((2, 2, 512), device="cuda")
    for _ in range(2):
        sv.attention_weight_sum(q.cuda(), a["k"], a["table"], a["seq_len"], lse, prior=w, out=w)
    # twice 3 rows of 4 heads, each of weight 1
    assert torch.allclose(w.double().sum(-1), torch.full((2, 2), 24.0, dtype=torch.float64,
                                                         device="cuda"), rtol=1e-4, atol=0)


def test_key_weights_of_bad_requests():
    cache = ref.Cache([100, 100, 100, 100], 16, 1, 64, torch.float16, seed=13)
    q = queries(4, 3, 2, 64, torch.float16)
    a = dev_args(cache, [2, 2, 2, 2])
    _, lse = sv.paged_attention(q.cuda(), a["k"], a["v"], a["table"], a["seq_len"])
    acc = torch.tensor([3, 1, 1, -1]).int().cuda()
    a["seq_len"][1] = -5
    a["table"][2, 3] = a["k"].shape[0] + 9
    w = sv.attention_weight_sum(q.cuda(), a["k"], a["table"], a["seq_len"], lse,
                                num_draft=a["num_draft"], accept_len=acc,
                                out=torch.full((4, 1, 112), 7.0, device="cuda")).cpu()
    assert math.isnan(w[0, 0, 0]) and bool((w[0, 0, 1:] == 7).all())
    assert math.isnan(w[1, 0, 0]) and bool((w[1, 0, 1:] == 7).all())
    nan = w[2, 0].isnan()
    assert bool(nan[48:64].all()) and not bool(nan[:48].any()) and not bool(nan[64:].any())
    assert bool((w[3, 0, :100] == 0).all()) and bool((w[3, 0, 100:] == 7).all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("G,P", [(4, 3), (8, 5), (16, 9)])
def test_rows_that_do_not_count_may_hold_anything(value, G, P):
    lens = [40, 130, 257, 300]
    cache = ref.Cache(lens, 16, 2, 64, torch.bfloat16, seed=31)
    nd, acc = [0, 1, P - 1, P - 1], [0, 0, 1, P - 2]
    q = queries(4, P, 2 * G, 64, torch.bfloat16)
    junk = q.clone()
    for b, n in enumerate(nd):
        junk[b, n + 1:] = value
    out, lse = check_attention(cache, junk, nd)
    for b, n in enumerate(acc):
        junk[b, n + 1:] = value
    a = dev_args(cache, nd)
    got = sv.attention_weight_sum(junk.cuda(), a["k"], a["table"], a["seq_len"], lse.cuda(),
                                  num_draft=a["num_draft"],
                                  accept_len=torch.tensor(acc).int().cuda(),
                                  out=torch.full((4, 2, 304), 7.0, device="cuda")).cpu()
    want, tol = ref.weight_sum(cache, q, nd, acc, lse, torch.zeros((4, 2, 304)),
                               scale=64 ** -0.5)
    for b, n in enumerate(lens):
        assert ref.close(got[b, :, :n], want[b, :, :n], tol[b, :, :n]), b


def test_a_cap_far_above_the_scores_changes_nothing():
    # c tanh(s / c) is s - s^3 / 3c^2: less than 2^-30 of a score of 100 at c = 10^7
    cache = ref.Cache([1, 200, 513], 16, 2, 128, torch.float16, seed=32)
    q = queries(3, 2, 8, 128, torch.float16)
    a = dev_args(cache, None)
    args = (q.cuda(), a["k"], a["v"], a["table"], a["seq_len"])
    out, lse = sv.paged_attention(*args)
    capped, lse_c = sv.paged_attention(*args, softcap=1e7)
    want = ref.attention(cache, q, [1, 1, 1], scale=128 ** -0.5)
    for b in range(3):
        for i in range(2):
            for head in range(8):
                if not (b == 0 and i == 0):  # (the row of a cache of one that sees no key)
                    o, l, tol, tol_l = want[b, i, head]
                    assert ref.close(capped[b, i, head].cpu(), o, tol), (b, i, head)
                    assert abs(float(lse_c[b, i, head]) - l) <= tol_l, (b, i, head)
    assert bool((lse_c[0, 0] == -math.inf).all())
