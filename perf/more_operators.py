"""Measured cases of a serving step over a cache held in 8 bits: the pages and slots of the new
positions, the norm and rotation of their queries and keys, the append that quantises keys and
values block by block, and the attention that reads them.

A case is a dict of plain values; ``prepare`` makes its inputs from a seed, ``run`` is one call (the
framework's kernels where ``own`` is true, elementary torch operations elsewhere), ``work`` the bytes
and operations the call cannot do without, and ``exact`` the definition in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CODE = torch.float8_e4m3fn
LARGEST = 448.0  # of the 8-bit type


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a verify step of a full batch: drafts were rejected, requests ended, others came in
        pages("map a verify step", B=512, P=9, lo=200, hi=16384, new=9, page=16, fresh=0.05),
        # admitted prompts of all lengths, packed row by row
        pages("map packed prompts", B=1024, P=0, lo=16, hi=16384, new=16384, page=16, fresh=0.9),
        # plain decoding of one request far into its context: latency
        rotate("rotate one token", B=1, P=1, Hq=32, Hkv=8, D=128, R=128, far=131072, dtype="bf16"),
        # the new positions of a verify batch
        rotate("rotate a verify batch", B=64, P=6, Hq=64, Hkv=8, D=128, R=64, far=16384,
               dtype="fp16", interleaved=True, weight="fp16"),
        # packed prompts
        rotate("rotate prompts", B=1, P=24576, Hq=32, Hkv=8, D=128, R=128, far=32768, dtype="bf16"),
        # one token of a batch: most land in a block that holds earlier tokens
        append("append one token of a batch", B=64, P=1, Hkv=8, D=128, lo=200, hi=8192, new=1,
               page=64, block=64, order="head", dtype="bf16"),
        # prompts of mixed lengths, behind cached prefixes
        append("append prompts", B=64, P=0, Hkv=8, D=128, lo=64, hi=8192, new=8192, page=32,
               block=32, order="token", dtype="bf16"),
        # plain decoding of one short conversation: latency
        attend("attend one token of one request", B=1, P=1, Hq=32, Hkv=8, D=128, lo=777, hi=777,
               page=16, block=16, order="token", dtype="bf16"),
        # plain decoding of a batch of mixed conversations
        attend("attend one token of a batch", B=64, P=1, Hq=32, Hkv=8, D=128, lo=200, hi=8192,
               page=64, block=64, order="head", dtype="bf16"),
        # verify of 5 drafts with wide groups: 48 query rows share each key
        attend("attend five drafts of a batch", B=32, P=6, Hq=64, Hkv=8, D=128, lo=500, hi=16384,
               page=32, block=32, order="token", dtype="fp16"),
        # verify of 8 drafts over two very long documents
        attend("attend eight drafts over long caches", B=2, P=9, Hq=32, Hkv=8, D=128, lo=100001,
               hi=131072, page=128, block=64, order="token", dtype="bf16"),
        # capped scores, a window, wide heads
        attend("attend capped scores in a window", B=16, P=5, Hq=16, Hkv=8, D=256, lo=100, hi=8192,
               page=16, block=16, order="head", dtype="bf16", softcap=50.0, window=4096),
    ]


def pages(name, *, B, P, lo, hi, new, page, fresh, short=False, ragged=1):
    return dict(name=name, op="pages", B=B, P=P, lo=lo, hi=hi, new=new, page=page, fresh=fresh,
                short=short, ragged=ragged)


def rotate(name, *, B, P, Hq, Hkv, D, R, far, dtype, interleaved=False, weight="fp32", ragged=1):
    return dict(name=name, op="rotate", B=B, P=P, Hq=Hq, Hkv=Hkv, D=D, R=R, far=far, dtype=dtype,
                interleaved=interleaved, weight=weight, ragged=ragged)


def append(name, *, B, P, Hkv, D, lo, hi, new, page, block, order, dtype, ragged=1):
    return dict(name=name, op="append", B=B, P=P, Hkv=Hkv, D=D, lo=lo, hi=hi, new=new, page=page,
                block=block, order=order, dtype=dtype, ragged=ragged)


def attend(name, *, B, P, Hq, Hkv, D, lo, hi, page, block, order, dtype, softcap=0.0, window=0,
           slopes=False, ragged=1):
    return dict(name=name, op="attend", B=B, P=P, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, page=page,
                block=block, order=order, dtype=dtype, softcap=softcap, window=window,
                slopes=slopes, ragged=ragged)


def draw(rng):
    most = {}
    for case in listed():
        w = work(case)
        top = most.setdefault(case["op"], {"bytes": 0.0, "flops": 0.0})
        top.update({k: max(top[k], w[k]) for k in top})
    op = rng.choice(["pages", "rotate", "append", "attend", "attend"])
    while True:
        case = _draw(rng, op)
        w = work(case)
        if all(w[k] <= most[op][k] for k in w):
            del case["name"]
            return case


def _draw(rng, op):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    ragged = rng.randrange(1, 1 << 30)
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    P = rng.randint(1, 9)
    if op == "pages":
        hi = log(64, 32768)
        packed = rng.random() < 0.5
        return pages("", B=log(1, 2048), P=0 if packed else P, lo=max(P, hi // rng.randint(1, 40)),
                     hi=hi, new=hi if packed else P, page=page, ragged=ragged,
                     fresh=rng.random() if packed else 0.1 * rng.random(),
                     short=rng.random() < 0.2)
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 2, 3, 4, 4, 7, 8])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rotate":
        packed = rng.random() < 0.4
        return rotate("", B=1 if packed else log(1, 512), P=log(1, 24576) if packed else P,
                      Hq=Hkv * G, Hkv=Hkv, D=D, R=D if rng.random() < 0.6 else 16 * rng.randint(1, D // 16),
                      far=log(100, 1 << 20), dtype=dtype, interleaved=rng.random() < 0.4,
                      weight=rng.choice(["fp32", dtype]), ragged=ragged)
    block = rng.choice([b for b in (1, 4, 16, 32, 64, 128) if b <= page])
    order = rng.choice(["token", "head"])
    if op == "append":
        packed = rng.random() < 0.5
        hi = log(64, 8192)
        return append("", B=log(1, 64), P=0 if packed else P, Hkv=Hkv, D=D,
                      lo=max(P, hi // rng.randint(1, 30)), hi=hi, new=hi if packed else P,
                      page=page, block=block, order=order, dtype=dtype, ragged=ragged)
    hi = log(64, 131072)
    return attend("", B=log(1, 64), P=P, Hq=Hkv * G, Hkv=Hkv, D=D, lo=max(9, hi // rng.randint(1, 30)),
                  hi=hi, page=page, block=block, order=order, dtype=dtype,
                  softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, 0, 500, 4096]),
                  slopes=rng.random() < 0.25, ragged=ragged)


def lengths(case):
    """Tokens in each request's cache: over the logarithm of [lo, hi], the longest in its place."""
    r = random.Random(case["ragged"])
    lo, hi = case["lo"], case["hi"]
    n = [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(case["B"])]
    n[r.randrange(case["B"])] = hi
    return n


def drafts(case):
    """Drafted tokens of each request: all P - 1 of most, fewer of some."""
    r = random.Random(case["ragged"] + 1)
    k = case["P"] - 1
    return [k if r.random() < 0.7 else r.randint(0, k) for _ in range(case["B"])]


def steps(case):
    """(tokens whose pages a request holds, tokens after the step, new ones among them) each."""
    r = random.Random(case["ragged"] + 4)
    found = []
    for n in lengths(case):
        u = r.random()
        if case["P"] == 0:  # a prompt, or the rest of one behind what is cached
            new = n if u < case["fresh"] else r.randint(1, n)
            found.append((n - new, n, new))
        elif u < case["fresh"]:  # ended, or the first tokens of another
            found.append((n, 0, 0) if r.random() < 0.5 else (0, case["P"], case["P"]))
        else:  # the rejected drafts of the last step go, the new positions come
            new = r.randint(1, case["P"])
            found.append((n, n - r.randint(0, min(n, case["P"]) - 1) + new, new))
    return found


def writes(case):
    """(tokens cached before, new ones) of each request of an append."""
    r = random.Random(case["ragged"] + 5)
    if case["P"]:
        return [(n, d + 1) for n, d in zip(lengths(case), drafts(case))]
    new = [r.randint(1, n) for n in lengths(case)]
    return [(n - x, x) for n, x in zip(lengths(case), new)]


def work(case):
    if case["op"] == "pages":
        page = case["page"]
        up = lambda n: -(-n // page)  # noqa: E731
        s = steps(case)
        rows = len(s) * case["P"] if case["P"] else sum(x for _, _, x in s)
        held = sum(min(up(a), up(b)) - (b - x) // page for a, b, x in s if up(a) > (b - x) // page and x)
        moved = sum(abs(up(b) - up(a)) for a, b, _ in s)
        return {"bytes": float(12 * rows + 4 * held + 8 * moved + 20 * len(s)), "flops": float(rows)}
    D, Hkv = case["D"], case["Hkv"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rotate":
        live = case["B"] * case["P"] if case["B"] == 1 else sum(d + 1 for d in drafts(case))
        heads = case["Hq"] + Hkv
        return {"bytes": float(2 * size * live * heads * D + 4 * case["B"] * case["P"]),
                "flops": float(live * heads * (4 * D + 3 * case["R"]))}
    if case["op"] == "append":
        rows = sum(x for _, x in writes(case))
        blocks = sum((n + x - 1) // case["block"] - n // case["block"] + 1 for n, x in writes(case))
        return {"bytes": float(2 * rows * Hkv * D * (size + 1) + 8 * rows + 8 * blocks * Hkv),
                "flops": float(4 * rows * Hkv * D)}
    G = case["Hq"] // Hkv
    keys = pairs = rows = 0
    for n, d in zip(lengths(case), drafts(case)):
        pos = [n - 1 - d + i for i in range(d + 1)]
        start = [max(0, p - case["window"] + 1) if case["window"] else 0 for p in pos]
        keys += n - min(start)
        pairs += sum(p + 1 - s for p, s in zip(pos, start))
        rows += d + 1
    return {"bytes": float(keys * Hkv * (2 * D + 8 / case["block"])
                           + rows * case["Hq"] * (2 * D * size + 4)),
            "flops": float(4 * D * pairs * Hkv * G)}


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    return {"pages": _prepare_pages, "rotate": _prepare_rotate, "append": _prepare_append,
            "attend": _prepare_attend}[case["op"]](case, g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(counts, width, ids):
    """A page table [B, width]: counts[b] pages each, taken from ids in order, then -1."""
    col = torch.arange(width, device="cuda")
    have = _ints(counts)[:, None].long()
    first = have.cumsum(0) - have
    at = (first + col).clamp(max=max(0, ids.numel() - 1))
    return torch.where(col < have, ids[at], torch.full_like(ids[at], -1))


def _prepare_pages(case, g):
    page, B = case["page"], case["B"]
    up = lambda n: -(-n // page)  # noqa: E731
    s = steps(case)
    held = [up(a) for a, _, _ in s]
    grown = sum(max(0, up(b) - up(a)) for a, b, _ in s)
    # a pool that runs dry has not enough for all of them
    total = sum(held) + (2 * grown // 3 if case["short"] else grown + 100) + 1
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(max(up(a), up(b)) for a, b, _ in s))
    # the free pages wait in a ring of places, from somewhere in it on
    free = total - sum(held)
    head = int(torch.randint(0, total, (1,), generator=g, device="cuda"))
    ring = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(free, device="cuda")) % total] = ids[sum(held):]
    rows = B * case["P"] if case["P"] else sum(x for _, _, x in s)
    return {"case": case, "table": _table(held, width, ids[:max(1, sum(held))]),
            "old_len": _ints([a for a, _, _ in s]), "seq_len": _ints([b for _, b, _ in s]),
            "num_new": _ints([x for _, _, x in s]), "ring": ring, "state": _ints([head, free]),
            "num_pages": total, "rows": rows,
            "slots": torch.zeros((B, case["P"]) if case["P"] else (rows,), dtype=torch.int64, device="cuda"),
            "positions": _ints([0] * rows).view((B, case["P"]) if case["P"] else (rows,)),
            "length": _ints([0] * B), "first": _ints([0] * (B + 1)), "next": _ints([0, 0])}


def _prepare_rotate(case, g):
    B, P, Hq, Hkv, D, R = (case[x] for x in ("B", "P", "Hq", "Hkv", "D", "R"))
    dtype = TYPES[case["dtype"]]
    # queries and keys lie side by side in the projection's rows; channels differ in size
    qkv = torch.randn((B, P, Hq + 2 * Hkv, D), generator=g, device="cuda", dtype=dtype)
    qkv *= torch.exp(0.5 * torch.randn((Hq + 2 * Hkv, D), generator=g, device="cuda")).to(dtype)
    start = torch.randint(0, case["far"], (B, 1), generator=g, device="cuda")
    positions = (start + torch.arange(P, device="cuda")).int()
    if B > 1:
        positions = torch.where(torch.arange(P, device="cuda") <= _ints(drafts(case))[:, None],
                                positions, -1)
    weights = 1 + 0.3 * torch.randn((2, D), generator=g, device="cuda")
    weights = weights.to(TYPES[case["weight"]])
    return {"case": case, "q": qkv[..., :Hq, :], "k": qkv[..., Hq:Hq + Hkv, :],
            "positions": positions, "q_weight": weights[0], "k_weight": weights[1],
            "inv_freq": 500000.0 ** (-torch.arange(0, R, 2, device="cuda").float() / R),
            "out_q": torch.zeros((B, P, Hq, D), dtype=dtype, device="cuda"),
            "out_k": torch.zeros((B, P, Hkv, D), dtype=dtype, device="cuda")}


def _scale_for(top):
    """The smallest power of two that brings a block's largest magnitude within the 8-bit type."""
    m, e = torch.frexp((top / LARGEST).clamp(min=2.0 ** -40))
    return torch.exp2((e - (m == 0.5).int()).float().clamp(max=40))


def _cached(case, total, g):
    """A pool of keys or values in 8 bits, [pages, page, Hkv, D] in one of two orders, with its
    scales [pages, blocks, Hkv]: tokens differ in size, and a few channels stand out."""
    page, block, Hkv, D = (case[x] for x in ("page", "block", "Hkv", "D"))
    size = torch.exp(0.4 * torch.randn((total, page, Hkv, 1), generator=g, device="cuda"))
    size = size * torch.exp(0.5 * torch.randn((1, 1, Hkv, D), generator=g, device="cuda"))
    x = torch.randn((total, page, Hkv, D), generator=g, device="cuda") * size
    top = x.abs().amax(-1).unflatten(1, (page // block, block)).amax(2)
    scale = _scale_for(top)
    codes = (x / scale.repeat_interleave(block, 1)[..., None]).to(CODE)
    del x, size
    if case["order"] == "head":
        codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
    return codes, scale


def _prepare_append(case, g):
    page, Hkv, D, dtype = case["page"], case["Hkv"], case["D"], TYPES[case["dtype"]]
    w = writes(case)
    counts = [-(-(n + x) // page) for n, x in w]
    total = sum(counts)
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = _table(counts, max(counts), ids)
    k_cache, k_scale = _cached(case, total, g)
    v_cache, v_scale = _cached(case, total, g)
    if case["P"]:
        col = torch.arange(case["P"], device="cuda")
        at = _ints([n for n, _ in w])[:, None].long() + col
        req = torch.arange(case["B"], device="cuda")[:, None].expand_as(at)
        live = col < _ints([x for _, x in w])[:, None]
        shape = at.shape
    else:
        new = _ints([x for _, x in w]).long()
        first = new.cumsum(0) - new
        row = torch.arange(sum(x for _, x in w), device="cuda")
        req = torch.searchsorted(first, row, right=True) - 1
        at = _ints([n for n, _ in w]).long()[req] + row - first[req]
        live = torch.ones_like(at, dtype=torch.bool)
        shape = row.shape
    slots = table[req, (at // page).clamp(max=table.shape[1] - 1)].long() * page + at % page
    slots = torch.where(live, slots, -1)
    # keys come from the norm and rotation, values as a slice of the projection's rows
    k = torch.randn((*shape, Hkv, D), generator=g, device="cuda", dtype=dtype)
    v = torch.randn((*shape, 2 * Hkv, D), generator=g, device="cuda", dtype=dtype)[..., Hkv:, :]
    return {"case": case, "k": k, "v": v, "slots": slots, "k_cache": k_cache, "v_cache": v_cache,
            "k_scale": k_scale, "v_scale": v_scale}


def _prepare_attend(case, g):
    B, P, Hq, Hkv, D, page = (case[x] for x in ("B", "P", "Hq", "Hkv", "D", "page"))
    n = lengths(case)
    counts = [-(-x // page) for x in n]
    s = {"case": case, "seq_len": _ints(n)}
    s["table"] = _table(counts, max(counts), torch.randperm(sum(counts), generator=g,
                                                            device="cuda").to(torch.int32))
    s["k"], s["k_scale"] = _cached(case, sum(counts), g)
    s["v"], s["v_scale"] = _cached(case, sum(counts), g)
    # the queries are a slice of the projection's rows, which hold keys and values too
    qkv = torch.randn((B, P, Hq + 2 * Hkv, D), generator=g, device="cuda", dtype=TYPES[case["dtype"]])
    s["q"] = qkv[..., :Hq, :]
    s["num_draft"] = _ints(drafts(case)) if P > 1 else None
    s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)
                   if case["slopes"] else None)
    s["scale"] = D ** -0.5
    s["out"] = torch.zeros((B, P, Hq, D), dtype=qkv.dtype, device="cuda")
    s["lse"] = torch.zeros((B, P, Hq), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state, state["case"])
    return _PLAIN[op](state, state["case"])


def _own_pages(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    made = sv.kv_page_map(
        s["table"], s["old_len"], s["seq_len"], s["num_new"], s["ring"], s["state"], case["page"],
        s["num_pages"], out_slots=s["slots"], out_positions=s["positions"], out_len=s["length"],
        out_first=s["first"], out_state=s["next"])
    return (*made, s["table"], s["ring"])


def _own_rotate(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    return sv.qk_norm_rotate(
        s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
        k_weight=s["k_weight"], eps=1e-6, interleaved=case["interleaved"], out_q=s["out_q"],
        out_k=s["out_k"])


def _own_append(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    sv.kv_cache_append_q8(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"],
                          s["v_scale"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _own_attend(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    return sv.paged_attention_q8(
        s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["seq_len"],
        num_draft=s["num_draft"], scale=s["scale"], softcap=case["softcap"], window=case["window"],
        slopes=s["slopes"], out=s["out"], out_lse=s["lse"])


def _plain_pages(s, case):
    """A request takes the pages it lacks from the ring's front, in order, as long as those before
    it and it find enough; the pages past its new length go to the ring's end."""
    page, B, P, rows = case["page"], case["B"], case["P"], s["rows"]
    table, ring, size = s["table"].clone(), s["ring"].clone(), s["ring"].numel()
    dev = table.device
    old, want, new = (s[x].long() for x in ("old_len", "seq_len", "num_new"))
    have, need = -(-old // page), -(-want // page)
    head, free = s["state"].long()
    grow, drop = (need - have).clamp(min=0), (have - need).clamp(min=0)
    fits = (grow == 0) | (grow.cumsum(0) <= free)
    grow = torch.where(fits, grow, 0)
    taken, given = grow.cumsum(0), drop.cumsum(0)
    t = torch.arange(table.shape[1], device=dev)
    source = (head + (taken - grow)[:, None] + t - have[:, None]) % size
    fresh = (t >= have[:, None]) & (t < (have + grow)[:, None])
    pages_of = torch.where(fresh, ring[source], table)
    # what is given back, in the order of the requests; the others land in a place that is cut off
    target = (head + free + (given - drop)[:, None] + t - need[:, None]) % size
    target = torch.where((t >= need[:, None]) & (t < have[:, None]), target, size)
    ring = torch.cat([ring, ring[:1]]).scatter_(0, target.flatten(), table.flatten())[:size]
    first = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    if P:
        first = P * torch.arange(B + 1, device=dev)
    row = torch.arange(rows, device=dev)
    req = (torch.searchsorted(first, row, right=True) - 1).clamp(max=B - 1)
    i = row - first[req]
    live = (i < new[req]) & fits[req]
    at = (want - new)[req] + i
    of = pages_of[req, (at // page).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(live & (of >= 0) & (of < s["num_pages"]), of * page + at % page, -1)
    positions = torch.where(live, at, -1).int()
    if P:
        slots, positions = slots.view(B, P), positions.view(B, P)
    state = torch.stack([(head + taken[-1]) % size, free - taken[-1] + given[-1]]).int()
    return slots, positions, torch.where(fits, want, old).int(), first.int(), state, pages_of, ring


def _plain_rotate(s, case):
    R = case["R"]
    # angles of far positions need more than 32 bits; their sines and cosines do not
    angle = s["positions"].double()[..., None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]
    live = (s["positions"] >= 0)[..., None, None]

    def one(x, weight, out):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        a, b = ((y[..., 0:R:2], y[..., 1:R:2]) if case["interleaved"]
                else (y[..., :R // 2], y[..., R // 2:R]))
        turned = (a * cos - b * sin, a * sin + b * cos)
        turned = torch.stack(turned, -1).flatten(-2) if case["interleaved"] else torch.cat(turned, -1)
        return torch.where(live, torch.cat([turned, y[..., R:]], -1).to(out.dtype), out)

    return one(s["q"], s["q_weight"], s["out_q"]), one(s["k"], s["k_weight"], s["out_k"])


def _plain_append(s, case):
    """Blocks of tokens have a scale each, a power of two that the new tokens can only raise;
    where they do, the block's earlier tokens are rounded again."""
    page, block, Hkv, D = (case[x] for x in ("page", "block", "Hkv", "D"))
    slots = s["slots"].flatten()
    row = torch.nonzero(slots >= 0).flatten()
    slots = slots[row]
    place, blocks = slots // block, s["k_scale"].shape[0] * (page // block)
    lowest = torch.full((blocks,), blocks * block, device=slots.device).scatter_reduce_(
        0, place, slots, "amin")
    touched = lowest < blocks * block
    # the block holds earlier tokens, those of its slots below the first new one
    slot = torch.arange(blocks * block, device=slots.device).view(blocks, block)
    earlier = (slot < lowest[:, None]) & touched[:, None]

    def one(new, cache, scale):
        x = new.flatten(0, -3)[row].float()
        top = torch.zeros((blocks, Hkv), device=x.device).scatter_reduce_(
            0, place[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        was = torch.where(earlier.any(1)[:, None], scale.view(blocks, Hkv), 0)
        now = torch.where(touched[:, None], torch.maximum(was, _scale_for(top)), scale.view(blocks, Hkv))
        ratio = torch.where(earlier[..., None], (scale.view(blocks, Hkv) / now)[:, None], 1)
        codes = cache.reshape(blocks, block, Hkv, D).float().contiguous()
        codes = (codes * ratio[..., None]).to(CODE).view(blocks * block, Hkv, D)
        codes[slots] = (x / now[place][..., None]).to(CODE)
        return codes.view(cache.shape), now.view(scale.shape)

    k, k_scale = one(s["k"], s["k_cache"], s["k_scale"])
    v, v_scale = one(s["v"], s["v_cache"], s["v_scale"])
    return k, v, k_scale, v_scale


def _gathered(pool, scale, table, n, block):
    """The pages of each request in a row: [B, Hkv, n, D] in 32 bits."""
    at = table.clamp(min=0).long()
    t = pool[at].float() * scale[at].repeat_interleave(block, 2)[..., None]  # [B, pages, page, Hkv, D]
    return t.flatten(1, 2)[:, :n].transpose(1, 2)


def _plain_attend(s, case):
    B, P, Hq, Hkv, D, n = (case[x] for x in ("B", "P", "Hq", "Hkv", "D", "hi"))
    G = Hq // Hkv
    q = s["q"].float().transpose(1, 2).reshape(B, Hkv, G * P, D)
    k = _gathered(s["k"], s["k_scale"], s["table"], n, case["block"])
    z = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, G, P, n)
    del k
    if case["softcap"]:
        z = torch.tanh(z / case["softcap"]) * case["softcap"]
    row = torch.arange(P, device="cuda")
    draft = (s["num_draft"] if s["num_draft"] is not None else torch.zeros_like(s["seq_len"]))[:, None]
    live = row <= draft
    pos = (s["seq_len"][:, None] - 1 - draft + row)[:, None, None, :, None]
    key = torch.arange(n, device="cuda")
    if s["slopes"] is not None:
        z = z - s["slopes"].view(1, Hkv, G, 1, 1) * (pos - key)
    sees = (key <= pos) & live[:, None, None, :, None]
    if case["window"]:
        sees = sees & (key > pos - case["window"])
    z = torch.where(sees, z, torch.full((), -math.inf, device="cuda"))
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z = (z - top).exp_()
    total = z.sum(-1, keepdim=True)
    v = _gathered(s["v"], s["v_scale"], s["table"], n, case["block"])
    o = torch.matmul(z.view(B, Hkv, -1, n), v).view(B, Hkv, G, P, D) / total
    o = o.reshape(B, Hq, P, D).transpose(1, 2).to(s["out"].dtype)
    lse = (top + total.log()).reshape(B, Hq, P).transpose(1, 2)
    return (torch.where(live[..., None, None], o, s["out"]),
            torch.where(live[..., None], lse, s["lse"]))


_OWN = {"pages": _own_pages, "rotate": _own_rotate, "append": _own_append, "attend": _own_attend}
_PLAIN = {"pages": _plain_pages, "rotate": _plain_rotate, "append": _plain_append,
          "attend": _plain_attend}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions, request by request, in 64 bits."""
    s = prepare(case, seed)
    return {"pages": _exact_pages, "rotate": _exact_rotate, "append": _exact_append,
            "attend": _exact_attend}[case["op"]](s, case)


def _exact_pages(s, case):
    page, P = case["page"], case["P"]
    table, ring = s["table"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    head, free = s["state"].tolist()
    at, end, left, size = head, head + free, free, ring.size
    slots, positions, length, first = [], [], [], [0]
    given = []
    asked = 0
    for b, (old, want, new) in enumerate(steps(case)):
        have, need = -(-old // page), -(-want // page)
        asked += max(0, need - have)
        fits = need <= have or asked <= free
        if need > have and fits:
            for t in range(have, need):
                table[b, t] = ring[at % size]
                at += 1
                left -= 1
        given += table[b, need:have].tolist()
        mine = [(int(table[b, p // page]) * page + p % page, p) for p in range(want - new, want)]
        mine = mine if fits else [(-1, -1)] * new
        mine += [(-1, -1)] * (P - new if P else 0)
        slots += [x for x, _ in mine]
        positions += [p for _, p in mine]
        length.append(want if fits else old)
        first.append(len(slots))
    for i, x in enumerate(given):
        ring[(end + i) % size] = x
    cuda = lambda v, t: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    slots, positions = cuda(slots, torch.int64), cuda(positions, torch.int32)
    if P:
        slots, positions = slots.view(-1, P), positions.view(-1, P)
    return (slots, positions, _ints(length), _ints(first), _ints([at % size, left + len(given)]),
            torch.from_numpy(table).cuda(), torch.from_numpy(ring).cuda())


def _exact_rotate(s, case):
    D, R = case["D"], case["R"]
    found = []
    for x, w, out in ((s["q"], s["q_weight"], s["out_q"]), (s["k"], s["k_weight"], s["out_k"])):
        res = out.double()
        norm = torch.linalg.vector_norm(x, dim=-1, dtype=torch.float64)
        shrink = 1 / torch.sqrt(norm * norm / D + 1e-6)
        for i in range(D):
            # the partner of component i, and which of the pair it is
            second = i < R and (i % 2 if case["interleaved"] else i >= R // 2)
            step = 1 if case["interleaved"] else R // 2
            value = x[..., i].double() * w[i].double()
            if i < R:
                j = i - step if second else i + step
                f = s["inv_freq"][i // 2 if case["interleaved"] else i % (R // 2)].double()
                angle = (s["positions"].double() * f)[..., None]
                other = x[..., j].double() * w[j].double()
                value = value * angle.cos() + (other if second else -other) * angle.sin()
            res[..., i] = torch.where((s["positions"] >= 0)[..., None], value * shrink, res[..., i])
        found.append(res)
    return tuple(found)


def _code(x):
    """The nearest value of the 8-bit type (ties to the even one), in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_append(s, case):
    page, block = case["page"], case["block"]
    if s["k_cache"].numel() > 3e8 or case["block"] * 60000 < s["slots"].numel():
        return None
    found, scales = [], []
    for new, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        codes, by = cache.double(), scale.double()
        x = new.flatten(0, -3)
        at = s["slots"].flatten()
        keep = at >= 0
        x, at = x[keep], at[keep]
        # the rows that start a block's run of new tokens
        cut = torch.nonzero(torch.diff(at // block, prepend=at.new_full((1,), -1))).flatten().tolist()
        for lo, hi in zip(cut, cut[1:] + [at.numel()]):
            slot = int(at[lo])
            p, first, b = slot // page, slot % page, slot % page // block
            rows = x[lo:hi].double()
            top = rows.abs().amax((0, 2)) / LARGEST
            now = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -40))))
            if first % block:
                now = torch.maximum(now, by[p, b])
                old = codes[p, b * block:first]
                codes[p, b * block:first] = _code(old * (by[p, b] / now)[:, None])
            by[p, b] = now
            codes[p, first:first + hi - lo] = _code(rows / now[:, None])
        found.append(codes)
        scales.append(by)
    return (*found, *scales)


def _cache_row(s, which, case, b, n):
    ids = s["table"][b, :-(-n // case["page"])].long()
    size = s[which + "_scale"][ids].double()[:, :, None].expand(-1, -1, case["block"], -1)
    return (s[which][ids].double() * size.flatten(1, 2)[..., None]).flatten(0, 1)[:n]  # [n, Hkv, D]


def _exact_attend(s, case):
    Hkv, D = case["Hkv"], case["D"]
    out, lse = s["out"].double(), s["lse"].double()
    for b, (n, d) in enumerate(zip(lengths(case), drafts(case))):
        q = s["q"][b, :d + 1].double().unflatten(1, (Hkv, -1))  # [rows, Hkv, G, D]
        z = torch.einsum("ihgd,jhd->hgij", q, _cache_row(s, "k", case, b, n)) / math.sqrt(D)
        if case["softcap"]:
            z = case["softcap"] * torch.tanh(z / case["softcap"])
        away = (n - 1 - d + torch.arange(d + 1, device="cuda"))[:, None] - torch.arange(n, device="cuda")
        if case["slopes"]:
            z -= s["slopes"].double().view(Hkv, -1, 1, 1) * away
        hidden = away < 0
        if case["window"]:
            hidden |= away >= case["window"]
        z = z.masked_fill(hidden, -math.inf)
        total = torch.logsumexp(z, -1)
        p = torch.exp(z - total[..., None])
        o = torch.einsum("hgij,jhd->ihgd", p, _cache_row(s, "v", case, b, n))
        out[b, :d + 1] = o.flatten(1, 2)
        lse[b, :d + 1] = total.flatten(0, 1).transpose(0, 1)
    return out, lse
