"""kv_cache_append_q8, kv_page_map and qk_norm_rotate against their definitions in 64 bits, and a step
that runs them with the attention over what they wrote."""
import math
import random

import pytest
import torch

import kv8_reference as ref8
import kv_reference as ref
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ append
def same(a, b):
    a, b = a.double().cpu(), b.double()
    return bool(((a == b) | a.isnan() & b.isnan()).all())


def run_append(x, slots, cache, *, strided=False, padded=None):
    """Appends rows x[0] (keys), x[1] (values) to a copy of a cache and checks all of it."""
    pools = [cache.view(w, "cuda").clone(memory_format=torch.preserve_format) for w in (0, 1)]
    scales = [s.cuda() for s in cache.scales]
    rows = [t.cuda() for t in x]
    if strided:
        T, H, D = rows[0].shape
        both = torch.zeros((T, 2 * H + 1, D + 8), dtype=rows[0].dtype, device="cuda")
        both[:, 1:H + 1, :D], both[:, H + 1:, :D] = rows[0], rows[1]
        rows = [both[:, 1:H + 1, :D], both[:, H + 1:, :D]]
    at = torch.tensor(slots, dtype=torch.int64, device="cuda")
    if padded:
        rows, at = [t.view(padded, -1, *t.shape[1:]) for t in rows], at.view(padded, -1)
    sv.kv_cache_append_q8(*rows, at, *pools, *scales)
    torch.cuda.synchronize()
    for w in (0, 1):
        codes, sc = ref8.append8(x[w], slots, cache.codes[w], cache.scales[w], cache.block)
        assert same(scales[w], sc)
        assert same(pools[w], codes)
    return pools, scales


def rows_of(cache, T, dtype, seed, spread=2.0):
    H = cache.codes[0].shape[2]
    g = torch.Generator().manual_seed(seed)
    make = lambda: (torch.randn((T, H, cache.D), generator=g)  # noqa: E731
                    * torch.exp(spread * torch.randn((T, H, 1), generator=g))).to(dtype)
    return make(), make()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,Hkv,page,block,order", [
    (64, 1, 8, 1, "token"), (64, 3, 16, 16, "head"), (128, 2, 64, 32, "token"),
    (128, 8, 256, 128, "head"), (256, 2, 32, 8, "token"), (256, 1, 1024, 64, "head"),
])
def test_appends_of_every_length(dtype, D, Hkv, page, block, order):
    """Requests that take 0 to 300 new tokens from anywhere in a block on, in packed rows."""
    r = random.Random(D + page)
    before = [0, 1, block - 1, block, page - 1, page, page + 3, 2 * page + block // 2, 77]
    new = [1, 0, 1, 2, 5, block, 2 * block + 1, 300, 9]
    cache = ref8.Cache8([a + b for a, b in zip(before, new)], page, block, Hkv, D, order=order, seed=page)
    slots = []
    for b, (n, x) in enumerate(zip(before, new)):
        slots += [int(cache.table[b, j // page]) * page + j % page for j in range(n, n + x)]
        if r.random() < 0.5:
            slots.append(-1)
        # what holds earlier tokens has scales; what lies past them is junk
    for w in (0, 1):
        cache.scales[w].nan_to_num_(0.25)
    run_append(rows_of(cache, len(slots), dtype, 3), slots, cache, strided=page % 32 == 0)


@pytest.mark.parametrize("P", [1, 4, 9])
def test_padded_rows_of_drafts(P):
    cache = ref8.Cache8([n + P for n in (3, 17, 40, 0, 63)], 16, 16, 2, 128, seed=P)
    nd = [P - 1, 0, P // 2, P - 1, P - 1]
    slots = []
    for b, n in enumerate((3, 17, 40, 0, 63)):
        slots += [int(cache.table[b, j // 16]) * 16 + j % 16 if j - n <= nd[b] else -1
                  for j in range(n, n + P)]
    for w in (0, 1):
        cache.scales[w].nan_to_num_(1.0)
    run_append(rows_of(cache, 5 * P, torch.bfloat16, 1), slots, cache, padded=5)


def test_token_by_token_equals_at_once():
    """Powers of two re-round earlier codes exactly, but for those that become subnormal."""
    n, page, block = 100, 32, 32
    cache = ref8.Cache8([n], page, block, 2, 128, seed=1, spare=0)
    x = rows_of(cache, n, torch.bfloat16, 5, spread=1.0)
    slots = [int(cache.table[0, j // page]) * page + j % page for j in range(n)]
    pools, scales = run_append(x, slots, cache)
    one = [cache.view(w, "cuda").clone() for w in (0, 1)]
    sc = [s.cuda() for s in cache.scales]
    for j in range(n):
        sv.kv_cache_append_q8(x[0][j:j + 1].cuda(), x[1][j:j + 1].cuda(),
                              torch.tensor(slots[j:j + 1], device="cuda"), *one, *sc)
    torch.cuda.synchronize()
    for w in (0, 1):
        blocks = -(-n // block)
        at = cache.table[0, :blocks].long().cuda()
        assert torch.equal(sc[w][at], scales[w][at])
        a = one[w][at].float().flatten(0, 1)[:n]
        b = pools[w][at].float().flatten(0, 1)[:n]
        # a subnormal code is a multiple of 2^-9, rounded twice at most
        assert bool(((a == b) | ((b.abs() < 2.0 ** -6) & ((a - b).abs() <= 2.0 ** -9))).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_that_no_code_stands_for(dtype):
    cache = ref8.Cache8([40, 20], 16, 8, 1, 64, seed=2)
    x = rows_of(cache, 4, dtype, 7)
    x[0][0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    x[0][1] = 0.0
    x[0][2] = math.nan
    x[1][3, 0, 5] = 3e38 if dtype == torch.bfloat16 else 65504.0
    x[1][0] = 2.0 ** -60
    slots = [int(cache.table[0, 0]) * 16 + i for i in (1, 2, 3, 8)]
    run_append(x, slots, cache)


@pytest.mark.parametrize("bad", [math.nan, -1.0, math.inf, 2.0 ** 41, 0.0])
def test_earlier_scales_that_are_none(bad):
    cache = ref8.Cache8([40], 16, 8, 2, 64, seed=3)
    page = int(cache.table[0, 1])
    for w in (0, 1):
        cache.scales[w][page, 0, 1] = bad
    run_append(rows_of(cache, 2, torch.float16, 1), [page * 16 + 5, page * 16 + 6], cache)


def test_slots_out_of_order_and_outside():
    cache = ref8.Cache8([64], 16, 8, 2, 64, seed=4)
    pages = cache.codes[0].shape[0]
    p = [int(x) * 16 for x in cache.table[0]]
    for slots in ([p[0] + 2, p[0] + 1], [p[0] + 3, p[0] + 3], [-5, 2 ** 40, pages * 16, p[1] + 1],
                  [p[1] + 4] * 40, [p[2] + 7, p[2] + 8, p[3], p[3] + 7], list(range(p[0], p[0] + 8)) * 20):
        run_append(rows_of(cache, len(slots), torch.bfloat16, 2), slots, cache)


# ------------------------------------------------------------------------------ page map
def run_map(table, olds, lens, add, ring, state, page, num_pages, P, rows, **kw):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t, g = i32(table), i32(ring)
    args = (t, i32(olds), i32(lens), i32(add), g, i32(state), page, num_pages)
    for _ in range(2):  # (a call does the same again)
        got = sv.kv_page_map(*args, **(dict(P=P) if P else dict(rows=rows)), **kw)
        torch.cuda.synchronize()
    table, ring = [list(x) for x in table], list(ring)
    want = ref8.page_map(table, olds, lens, add, ring, state, page, num_pages, P, rows)
    assert got[0].flatten().tolist() == want[0]
    assert got[1].flatten().tolist() == want[1]
    assert got[2].tolist() == want[2]
    assert got[3].tolist() == want[3]
    assert got[4].tolist() == list(want[4])
    assert t.tolist() == table and g.tolist() == ring
    return want


def world(r, B, page, cols, spare, size=None):
    """Requests that hold pages, and a ring of the others."""
    olds = [r.choice([0, r.randint(0, cols * page), r.randint(0, 3 * page), page * r.randint(0, cols)])
            for _ in range(B)]
    olds = [min(x, cols * page) for x in olds]
    held = [-(-x // page) for x in olds]
    total = sum(held) + spare
    ids = list(range(total))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (cols - h))
        at += h
    size = total + (size or 0)
    head = r.randrange(max(1, size))
    ring = [-7] * max(1, size)
    for i, x in enumerate(ids[at:]):
        ring[(head + i) % size] = x
    return olds, table, ring, [head, spare], total


@pytest.mark.parametrize("B,page,cols,spare,P", [
    (1, 8, 3, 4, 1), (1, 16, 1, 0, 5), (5, 16, 40, 3, 4), (7, 64, 9, 100, 0), (300, 8, 20, 40, 9),
    (300, 32, 30, 10 ** 4, 0), (513, 16, 6, 700, 3), (2000, 8, 12, 3000, 0), (8192, 8, 4, 5000, 2),
])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_pages_and_slots(B, page, cols, spare, P, seed):
    r = random.Random(seed * 1000 + B)
    olds, table, ring, state, total = world(r, B, page, cols, spare, size=r.choice([0, 5]))
    lens, add = [], []
    for n in olds:
        m = r.choice([0, n, min(cols * page, n + r.randint(1, 2 * page)), r.randint(0, cols * page)])
        lens.append(m)
        add.append(r.randint(0, min(m, P) if P else min(m, 200)))
    rows = B * P if P else sum(add) + r.choice([0, 0, 7, -3])
    run_map(table, olds, lens, add, ring, state, page, max(0, total - seed), P, max(0, rows))


def test_data_errors_of_requests_and_of_the_ring():
    r = random.Random(5)
    olds, table, ring, state, total = world(r, 12, 16, 8, 30)
    lens = [min(128, n + 5) for n in olds]
    add = [min(4, n) for n in lens]
    for at, (a, n, x) in {1: (-1, 5, 1), 3: (129, 20, 1), 5: (olds[5], 129, 1), 6: (olds[6], -3, 0),
                          8: (olds[8], lens[8], -1), 9: (olds[9], 3, 4), 11: (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)}.items():
        olds[at], lens[at], add[at] = a, n, x
    run_map(table, olds, lens, add, ring, state, 16, total, 4, 48)
    run_map(table, olds, lens, add, ring, state, 16, total, 0, 48)
    for bad in ([-1, 3], [len(ring), 3], [0, -1], [0, len(ring) + 1], [2, len(ring)]):
        back = [0] * 12  # with pages to give back, the full ring has no room for them
        run_map(table, olds, back, back, ring, bad, 16, total, 4, 48)


def test_a_map_into_given_outputs_on_a_stream_and_in_a_graph():
    r = random.Random(6)
    olds, table, ring, state, total = world(r, 40, 16, 8, 200)
    lens = [min(128, n + 20) for n in olds]
    add = [min(3, n) for n in lens]
    st = torch.cuda.Stream()
    want = run_map(table, olds, lens, add, ring, state, 16, total, 3, 120, stream=st)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32(table), i32(olds), i32(lens), i32(add), i32(ring), i32(state), 16, total)
    odd = torch.zeros(121, dtype=torch.int64, device="cuda")[1:]  # off the 16-byte grid
    pos = torch.zeros(121, dtype=torch.int32, device="cuda")[1:]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.kv_page_map(*args, out_slots=odd.view(40, 3), out_positions=pos.view(40, 3))
    odd.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert odd.tolist() == want[0] and pos.tolist() == want[1] and got[2].tolist() == want[2]


# ------------------------------------------------------------------------------ norm and rotation
def run_rotate(q, k, positions, inv_freq, qw, kw, *, eps=1e-6, norm=True, interleaved=False, in_place=False,
               lead=None):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    shape = lambda t: t.cuda().view(*lead, *t.shape[1:]) if lead else t.cuda()  # noqa: E731
    qd, kd = shape(q), shape(k)
    outs = (qd, kd) if in_place else tuple(torch.full_like(t, 7.0) for t in (qd, kd))
    got = sv.qk_norm_rotate(qd, kd, shape(positions), d(inv_freq), q_weight=d(qw), k_weight=d(kw), eps=eps,
                            norm=norm, interleaved=interleaved, out_q=outs[0], out_k=outs[1])
    torch.cuda.synchronize()
    live = positions >= 0
    for x, w, g in ((q, qw, got[0]), (k, kw, got[1])):
        freq = torch.zeros(0) if inv_freq is None else inv_freq
        want, tol = ref8.norm_rotate(x, positions, freq, w, eps, norm, interleaved)
        g = g.cpu().view(x.shape)
        assert ref.close(g[live], want[live], tol[live])
        assert torch.equal(g[~live], x[~live] if in_place else torch.full_like(x, 7.0)[~live])


def heads(T, Hq, Hkv, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k = ((rand(T, H, D) * torch.exp(rand(T, H, 1))).to(dtype) for H in (Hq, Hkv))
    return q, k, 1 + 0.3 * rand(D), 1 + 0.3 * rand(D), g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R", [
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 7, 1, 128, 64), (9, 16, 8, 256, 256), (33, 5, 5, 64, 16),
    (130, 8, 2, 256, 48), (2500, 3, 1, 128, 128), (1300, 4, 4, 64, 32), (7, 9, 3, 128, 0),
])
def test_rows_of_heads(dtype, interleaved, T, Hq, Hkv, D, R):
    q, k, qw, kw, g = heads(T, Hq, Hkv, D, dtype)
    pos = torch.randint(0, 5000, (T,), generator=g).int()
    if T > 2:
        pos[1::4] = -1
        pos[2] = 0
    freq = 10000.0 ** (-torch.arange(R // 2) * 2.0 / R) if R else None
    weights = (qw, kw) if D != 64 else (qw.to(dtype), None)
    run_rotate(q, k, pos, freq, *weights, interleaved=interleaved, in_place=T == 33)


@pytest.mark.parametrize("freq64", [False, True])
def test_far_positions(freq64):
    q, k, _, _, g = heads(6, 4, 2, 128, torch.float16)
    pos = torch.tensor([131071, 10 ** 6, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, 99999]).int()
    freq = 500000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    run_rotate(q, k, pos, freq if freq64 else freq.float(), None, None)


def test_without_norm_and_with_large_frequencies():
    q, k, qw, kw, g = heads(20, 6, 2, 128, torch.bfloat16)
    pos = torch.randint(0, 100, (20,), generator=g).int()
    run_rotate(q, k, pos, torch.rand(32, generator=g) * 50 - 25, qw, kw, norm=False, lead=(4, 5))
    run_rotate(q, k, pos, torch.rand(64, generator=g), None, kw, eps=0.5, lead=(20, 1))


def test_rows_that_are_zero_or_not_finite():
    q, k, qw, kw, _ = heads(4, 2, 1, 64, torch.bfloat16)
    q[0], q[1, 0, 3], q[2, 1, 63] = 0.0, math.nan, math.inf
    pos = torch.arange(4).int()
    out, _ = sv.qk_norm_rotate(q.cuda(), k.cuda(), pos.cuda(), torch.ones(16).cuda())
    out = out.cpu()
    assert bool((out[0] == 0).all()) and bool(out[1, 0].isnan().all()) and not bool(out[1, 1].isnan().any())
    assert bool(out[2, 1].isnan().any()) and not bool(out[2, 0].isnan().any())


def test_slices_of_a_projection():
    g = torch.Generator(device="cuda").manual_seed(2)
    qkv = torch.randn((3, 5, 4 + 2 + 2, 128), generator=g, device="cuda").bfloat16()
    pos = torch.arange(15, device="cuda").int().view(3, 5)
    freq = torch.rand(64, generator=g, device="cuda")
    q, k = qkv[:, :, :4], qkv[:, :, 4:6]
    want = sv.qk_norm_rotate(q.contiguous(), k.contiguous(), pos, freq)
    got = sv.qk_norm_rotate(q, k, pos, freq)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    third = sv.qk_norm_rotate(q, k, pos, freq, stream=st)
    torch.cuda.synchronize()
    before = qkv.clone()
    sv.qk_norm_rotate(q, k, pos, freq, out_q=q, out_k=k)  # in place, the values beside them kept
    for a, b, c, d in zip(want, got, third, (q, k)):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
    assert torch.equal(before[:, :, 6:], qkv[:, :, 6:])


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_steps_of_a_batch(dtype):
    """Requests come, draft, reject and leave; every step's attention over the 8-bit cache is that of
    the rotated keys and values it was given, to the rounding of their codes."""
    r, g = random.Random(3), torch.Generator(device="cuda").manual_seed(3)
    B, P, Hq, Hkv, D, page, block, cols, total = 5, 4, 8, 2, 128, 16, 16, 12, 40
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    codes = [torch.zeros((total, page, Hkv, D), dtype=ref8.CODE, device="cuda") for _ in range(2)]
    scales = [torch.ones((total, page // block, Hkv), device="cuda") for _ in range(2)]
    table, ring, state = torch.full((B, cols), -1, dtype=torch.int32, device="cuda"), i32(list(range(total))), i32([0, total])
    freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    held, kept, history = [0] * B, [0] * B, [[] for _ in range(B)]
    for step in range(12):
        add = [r.randint(1, P) for _ in range(B)]
        for b in range(B):
            if r.random() < 0.1:  # the request ends, another takes its place
                kept[b], history[b] = 0, []
        lens = [k + a for k, a in zip(kept, add)]
        slots, pos, length, _, state = sv.kv_page_map(table, i32(held), i32(lens), i32(add), ring, state, page,
                                                      total, P=P)
        assert length.tolist() == lens
        q, k, v = (torch.randn((B, P, H, D), generator=g, device="cuda").to(dtype) for H in (Hq, Hkv, Hkv))
        q, k = sv.qk_norm_rotate(q, k, pos, freq, eps=1e-5)
        sv.kv_cache_append_q8(k, v, slots, *codes, *scales)
        nd = i32([a - 1 for a in add])
        out, lse = sv.paged_attention_q8(q, *codes, *scales, table, length, num_draft=nd)
        torch.cuda.synchronize()
        for b in range(B):
            history[b] = history[b][:kept[b]] + [(k[b, i], v[b, i]) for i in range(add[b])]
        # the attention's definition over the codes as they lie there
        cache = ref8.Cache8.__new__(ref8.Cache8)
        cache.lens, cache.page, cache.block, cache.D = lens, page, block, D
        cache.table, cache.codes, cache.scales = table.cpu(), [c.cpu() for c in codes], [s.cpu() for s in scales]
        want, want_lse, tol, tol_lse = ref8.attention8(cache, q.cpu(), nd.tolist(), scale=D ** -0.5)
        live = torch.arange(P) <= nd.cpu()[:, None]
        assert ref.close(out.cpu()[live], want[live], tol[live])
        assert ref.close(lse.cpu()[live], want_lse[live], tol_lse[live])
        # and the codes stand for what was appended: half a step of 2^-3, and where codes are subnormal
        # half of 2^-9 of the scale, once for each power of two that the scale has risen by
        for b in range(B):
            at = cache.table[b].long().repeat_interleave(page)[:lens[b]]
            for w in (0, 1):
                x = torch.stack([y[w] for y in history[b]]).double().cpu()
                size = cache.scales[w][at].double().amax(1)[..., None]
                assert ref.close(torch.stack([cache.row(w, b, h) for h in range(Hkv)], 1), x,
                                 2.0 ** -4 * x.abs() + 2.0 ** -9 * size)
        held = lens
        kept = [n - r.randint(0, a - 1) for n, a in zip(lens, add)]  # rejected drafts leave
    in_use = sum(-(-n // page) for n in held)
    assert int(state[1]) == total - in_use
    names = [int(x) for b in range(B) for x in table[b, :-(-held[b] // page)]]
    free = [int(ring[(int(state[0]) + i) % total]) for i in range(int(state[1]))]
    assert sorted(names + free) == list(range(total))
