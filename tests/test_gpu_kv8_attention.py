"""paged_attention_q8 against its definition in 64 bits, where it can go wrong: lengths of zero and
one and around the tiles' edges, ragged drafts, pages and blocks that end inside a tile, slots past the
end that hold NaN, scales far apart, windows, masks that leave rows empty, bad pages, counts and scales,
NaN codes, strides, streams, graphs and bounded waits."""
import ctypes
import math

import pytest
import torch

import kv8_reference as ref8
import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv
from speculative_decoding_verification_17_gb300 import _native

pytestmark = pytest.mark.gpu


def queries(B, P, Hq, D, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + 99)
    return (torch.randn((B, P, Hq, D), generator=g) * size).to(dtype)


def call(cache, q, num_draft, *, out=None, lse=None, **rule):
    """(out, lse) on the CPU, from outputs that held 7."""
    B, P, Hq, D = q.shape
    out = torch.full((B, P, Hq, D), 7.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((B, P, Hq), 7.0, device="cuda") if lse is None else lse
    nd = None if num_draft is None else torch.tensor(num_draft).int().cuda()
    if rule.get("slopes") is not None:
        rule["slopes"] = rule["slopes"].cuda()
    sv.paged_attention_q8(q.cuda(), cache.view(0, "cuda"), cache.view(1, "cuda"), cache.scales[0].cuda(),
                          cache.scales[1].cuda(), cache.table.cuda(), cache.seq_len.cuda(), num_draft=nd,
                          out=out, out_lse=lse, **rule)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check(cache, q, num_draft, *, scale=None, **rule):
    B, P, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out, lse = call(cache, q, num_draft, scale=scale, **rule)
    nd = num_draft if num_draft is not None else [P - 1] * B
    want, want_lse, tol, tol_lse = ref8.attention8(cache, q, nd, scale=scale, **rule)
    live = torch.arange(P) <= torch.tensor(nd)[:, None]
    assert bool((out[~live] == 7).all()) and bool((lse[~live] == 7).all())
    assert ref.close(lse[live], want_lse[live], tol_lse[live])
    assert ref.close(out[live], want[live], tol[live])
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,Hq,Hkv,P,page,block,order", [
    (64, 4, 4, 1, 16, 16, "token"), (64, 8, 2, 3, 8, 1, "head"), (128, 8, 2, 1, 16, 4, "head"),
    (128, 14, 2, 4, 64, 32, "token"), (256, 4, 2, 2, 32, 32, "token"), (256, 2, 1, 5, 256, 128, "head"),
    (128, 6, 1, 17, 128, 64, "token"), (64, 32, 1, 9, 512, 2, "head"), (256, 16, 2, 5, 64, 8, "head"),
])
def test_lengths_and_layouts(dtype, D, Hq, Hkv, P, page, block, order):
    lens = [0, 1, 2, P, 63, 64, 65, 127, 128, 129, 200, 257, 391]
    nd = [min(P - 1, b % P) for b in range(len(lens))]
    cache = ref8.Cache8(lens, page, block, Hkv, D, order=order, seed=D + P)
    check(cache, queries(len(lens), P, Hq, D, dtype), nd)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rule", [
    dict(softcap=5.0), dict(window=1), dict(window=100), dict(window=130, softcap=20.0),
    dict(slopes=True), dict(slopes=True, window=64, softcap=3.0), dict(scale=0.0), dict(scale=-0.3),
])
def test_rules(D, rule):
    rule = dict(rule)
    if rule.get("slopes"):
        rule["slopes"] = torch.tensor([0.5, 0.0, -0.01, 0.1])
    cache = ref8.Cache8([5, 130, 300, 513], 16, 8, 2, D, seed=1)
    check(cache, queries(4, 4, 4, D, torch.bfloat16, size=2.0), [3, 0, 2, 3], **rule)


@pytest.mark.parametrize("spread,plain", [(0.0, True), (4.0, True), (8.0, False), (20.0, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scales_far_apart(spread, plain, dtype):
    """Blocks whose values are millions of times smaller or larger than others'."""
    cache = ref8.Cache8([700, 31, 1500], 32, 8, 2, 128, seed=4, spread=spread, plain_scales=plain)
    for s in cache.scales:
        s.clamp_(2.0 ** -39, 2.0 ** 39)
    for k in (0,):  # keys of that spread would leave one key's weight only
        cache.scales[k].clamp_(2.0 ** -9, 2.0 ** -5)
    check(cache, queries(3, 3, 8, 128, torch.bfloat16 if spread > 3 else dtype), [2, 1, 0])


def test_blocks_of_scale_zero():
    cache = ref8.Cache8([300, 40], 16, 4, 1, 64, seed=6)
    cache.scales[1][:, 1::2] = 0.0
    cache.scales[0][:, 2] = 0.0
    check(cache, queries(2, 2, 4, 64, torch.float16), [1, 1])
    cache.scales[1].zero_()
    out, _ = check(cache, queries(2, 2, 4, 64, torch.float16), [1, 1])
    assert bool((out == 0).all())


def test_long_caches_are_split_and_joined():
    cache = ref8.Cache8([3001, 17, 5000], 64, 64, 1, 128, seed=2)
    check(cache, queries(3, 2, 4, 128, torch.bfloat16, size=3.0), [1, 1, 0])


@pytest.mark.parametrize("D,Hq", [(64, 48), (128, 40), (256, 32)])
def test_many_rows_of_one_head(D, Hq):
    """More query rows per kv head than one pass holds."""
    cache = ref8.Cache8([150, 40], 16, 16, 1, D, seed=3)
    check(cache, queries(2, 9, Hq, D, torch.float16), [8, 5])


def test_queries_of_any_size():
    """Rows from 2^-120 to 2^100, with elements far below their row's largest, zero rows among them."""
    cache = ref8.Cache8([90, 33], 16, 16, 2, 128, seed=7)
    q = queries(2, 3, 4, 128, torch.float32)
    q[..., ::3] *= 2.0 ** -12
    q[..., 1::7] = 0.0
    q[1, 0, 0] = 0.0
    q[0, 1] *= 2.0 ** -10
    check(cache, q.to(torch.float16), [2, 2])
    q[0, 0, 0] *= 2.0 ** -120
    check(cache, q.to(torch.bfloat16), [2, 2])
    q[0, 2, 1] *= 2.0 ** 100  # one key takes all
    out, _ = call(cache, q.to(torch.bfloat16), [2, 2])
    s = cache.row(0, 0, 0) @ q.to(torch.bfloat16)[0, 2, 1].double()
    v = cache.row(1, 0, 0)[int(s.argmax())]
    assert ref.close(out[0, 2, 1], v, 2.0 ** -7 * v.abs())


def test_small_weights_count():
    """One key holds half of the weight, thousands of others the rest."""
    n = 4097
    cache = ref8.Cache8([n], 64, 64, 1, 64, seed=8, spread=0.0)
    k, v = cache.codes
    k.zero_()
    first = int(cache.table[0, 0])
    k[first, 0, 0, 0] = 1.0  # the oldest key
    cache.scales[0].fill_(1.0)
    x = torch.ones((1, 1, 4, 64))
    x[..., 0] = torch.tensor([8.3125, 0.0, 16.625, 18.0])
    for dtype in (torch.bfloat16, torch.float16):
        check(cache, x.to(dtype), None, scale=1.0)


def test_nan_codes_reach_the_rows_that_see_them_alone():
    cache = ref8.Cache8([200, 130, 20], 16, 16, 2, 128, seed=9)
    q = queries(3, 5, 4, 128, torch.bfloat16)
    nd = [4, 4, 3]
    for b, j, h, d in ((0, 198, 0, 5), (0, 3, 1, 127), (1, 129, 1, 64), (2, 19, 0, 0)):
        page = int(cache.table[b, j // 16])
        cache.codes[1].view(torch.uint8)[page, j % 16, h, d] = 0xff if d else 0x7f
    check(cache, q, nd)
    check(cache, q, nd, window=3)
    # a NaN key makes the whole row NaN, of the rows that see it
    page = int(cache.table[0, 199 // 16])
    cache.codes[0].view(torch.uint8)[page, 199 % 16, 1, 7] = 0x7f
    out, lse = call(cache, q, nd)
    assert bool(out[0, 4, 2:].isnan().all()) and bool(lse[0, 4, 2:].isnan().all())
    assert not bool(lse[0, :4].isnan().any()) and not bool(lse[0, 4, :2].isnan().any())


@pytest.mark.parametrize("which,bad", [(0, math.nan), (0, math.inf), (1, math.nan), (1, -1.0),
                                       (1, math.inf), (1, 2.0 ** 41)])
@pytest.mark.parametrize("j", [199, 5])
def test_bad_scales_reach_the_rows_that_see_them_alone(which, bad, j):
    cache = ref8.Cache8([200, 130], 16, 1, 2, 64, seed=10)
    q = queries(2, 3, 4, 64, torch.float16)
    good, good_lse = check(cache, q, [2, 2])
    cache.scales[which][int(cache.table[0, j // 16]), j % 16, 1] = bad
    out, lse = call(cache, q, [2, 2])
    rows = torch.zeros((2, 3, 4), dtype=torch.bool)
    rows[0, 2 if j == 199 else slice(None), 2:] = True
    assert bool(out[rows].isnan().all()) and bool(lse[rows].isnan().all())
    assert torch.equal(out[~rows], good[~rows]) and torch.equal(lse[~rows], good_lse[~rows])


def test_queries_that_are_not_finite():
    cache = ref8.Cache8([200, 130], 16, 16, 2, 128, seed=11)
    for dtype in (torch.bfloat16, torch.float16):
        q = queries(2, 3, 4, 128, dtype)
        good, _ = call(cache, q, [2, 1])
        q[0, 1, 2, 77], q[1, 0, 0, 0], q[1, 2] = math.inf, math.nan, math.nan  # (the last is not live)
        out, lse = call(cache, q, [2, 1])
        rows = torch.zeros((2, 3, 4), dtype=torch.bool)
        rows[0, 1, 2] = rows[1, 0, 0] = True
        assert bool(out[rows].isnan().all()) and bool(lse[rows].isnan().all())
        assert torch.equal(out[~rows], good[~rows])


def test_bad_counts_and_pages():
    cache = ref8.Cache8([200, 130, 50, 60, 70], 16, 4, 1, 64, seed=12)
    q = queries(5, 3, 4, 64, torch.bfloat16)
    good, _ = check(cache, q, [2, 2, 2, 2, 2])
    cache.seq_len[1] = 16 * cache.max_pages + 1
    cache.table[2, 1] = 10 ** 6
    cache.table[3, 3] = -1
    out, lse = call(cache, q, [2, 2, 2, 2, 5])
    for b in (1, 4):
        assert bool(out[b].isnan().all()) and bool(lse[b].isnan().all())
    assert bool(out[2].isnan().all()) and bool(out[3].isnan().all())
    assert torch.equal(out[0], good[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,G,P,page,block,rule", [
    (64, 1, 1, 16, 16, {}), (64, 5, 5, 8, 2, {}), (64, 8, 6, 64, 64, dict(window=300)),
    (128, 4, 1, 16, 16, dict(softcap=20.0)), (128, 4, 6, 128, 64, {}), (128, 8, 6, 32, 32, {}),
    (128, 16, 8, 256, 128, dict(slopes=True)), (256, 2, 3, 16, 1, {}), (256, 4, 7, 64, 16, {}),
    (256, 8, 6, 16, 16, dict(window=129)),
])
def test_many_requests_share_the_ranges(dtype, D, G, P, page, block, rule):
    """Every width of the kernel with far more pieces than CTAs, short and long caches side by side;
    twice, with equal bits."""
    g = torch.Generator().manual_seed(D + G + P)
    B, Hkv = 150, 2
    lens = torch.cat([torch.tensor([0, 1, P, 128, 129]),
                      torch.exp(torch.rand(B - 5, generator=g) * 7.6).int().clamp(1, 2000)]).int()
    lens = lens[torch.randperm(B, generator=g)].tolist()
    nd = torch.randint(0, P, (B,), generator=g).tolist()
    cache = ref8.Cache8(lens, page, block, Hkv, D, seed=5)
    rule = dict(rule)
    if rule.get("slopes"):
        rule["slopes"] = torch.rand(Hkv * G, generator=g) * 0.1
    q = queries(B, P, Hkv * G, D, dtype)
    out, lse = check(cache, q, nd, **rule)
    again, lse2 = call(cache, q, nd, scale=D ** -0.5, **rule)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_strides_streams_and_graphs():
    """Queries as a slice of a projection, a pool as a slice of a larger one, another stream, and two
    graphs captured one after the other and replayed at once."""
    cache = ref8.Cache8([400, 90, 800], 32, 16, 2, 128, seed=13)
    qkv = torch.randn((3, 4, 8 + 4, 128), generator=torch.Generator().manual_seed(3)).bfloat16()
    q = qkv[:, :, 2:10]
    want, want_lse = check(cache, q.contiguous(), [3, 2, 0])
    wide = torch.zeros((cache.codes[0].shape[0], 32, 3, 256), dtype=ref8.CODE, device="cuda")
    pools = []
    for which in (0, 1):
        w = wide.clone()
        w[:, :, :2, 64:192] = cache.view(which, "cuda")
        pools.append(w[:, :, :2, 64:192])
    nd = torch.tensor([3, 2, 0]).int().cuda()
    args = (qkv.cuda()[:, :, 2:10], *pools, cache.scales[0].cuda(), cache.scales[1].cuda(),
            cache.table.cuda(), cache.seq_len.cuda())
    live = (torch.arange(4) <= torch.tensor([3, 2, 0])[:, None])

    def same(out, lse):
        assert torch.equal(out.cpu()[live], want[live]) and torch.equal(lse.cpu()[live], want_lse[live])

    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = sv.paged_attention_q8(*args, num_draft=nd, stream=st)
    torch.cuda.synchronize()
    same(*got)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = sv.paged_attention_q8(*args, num_draft=nd)
        graphs.append((g, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, outs, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, outs, _ in graphs:
        same(*outs)


@pytest.mark.parametrize("us", [1, 2, 4, 10, 40])
@pytest.mark.parametrize("D,G,P,page,block,dtype", [
    (128, 4, 1, 64, 64, torch.bfloat16), (128, 8, 6, 16, 16, torch.float16),
    (64, 8, 9, 32, 8, torch.bfloat16), (256, 2, 3, 128, 32, torch.bfloat16)])
def test_rows_of_a_cta_that_gives_up_are_nan(D, G, P, page, block, dtype, us):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 3000, (30,), generator=g).tolist()
    lens[::5], lens[2] = [0] * 6, 5000
    cache = ref8.Cache8(lens, page, block, 2, D, seed=2)
    nd = torch.randint(0, P, (30,), generator=g).tolist()
    q = queries(30, P, 2 * G, D, dtype)
    want, want_lse = call(cache, q, nd)
    k, v, ks, vs = cache.view(0, "cuda"), cache.view(1, "cuda"), cache.scales[0].cuda(), cache.scales[1].cuda()
    table, n, ndt, qd = cache.table.cuda(), cache.seq_len.cuda(), torch.tensor(nd).int().cuda(), q.cuda()
    shape = _native.KvShape(1 if dtype == torch.bfloat16 else 2, 30, P, 2 * G, 2, D, page, k.shape[0],
                            table.shape[1])
    rule = _native.ScoreRule(D ** -0.5, 0.0, 0, None)
    pool = lambda t: ctypes.byref(_native.KvPool(t.data_ptr(), *t.stride()[:3]))  # noqa: E731
    L = sv.library()
    out, lse = torch.full_like(qd, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    ws = torch.full((L.paged_attention_q8_workspace(ctypes.byref(shape)),), 5, dtype=torch.uint8, device="cuda")
    status = L.paged_attention_q8_wait_selftest(
        ctypes.byref(shape), ctypes.byref(rule), qd.data_ptr(), *qd.stride()[:3], pool(k), pool(v),
        ks.data_ptr(), vs.data_ptr(), block, table.data_ptr(), n.data_ptr(), ndt.data_ptr(),
        out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), us,
        torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()
    out, lse = out.cpu(), lse.cpu()
    live = torch.arange(P) <= torch.tensor(nd)[:, None]
    assert bool(((out == want) | out.isnan() & live[..., None, None]).all())
    assert bool(((lse == want_lse) | lse.isnan()).all())
    # the device is as usable as before
    again, _ = call(cache, q, nd)
    assert torch.equal(again, want)
