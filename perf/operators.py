"""Measured cases of the operators around the verify step: the logits' penalties and masks, the
paged attention of the new positions, the weight each cached key received, and the eviction that
keeps the heaviest keys.

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


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one interactive request of a vocabulary that no vector width divides: latency
        adjust("adjust one request", B=1, P=5, V=50257, dtype="fp32", H=700, bias=12, mask=False),
        # the small verify batch, chat histories, half of the requests under a grammar
        adjust("adjust a small batch", B=64, P=6, V=32000, dtype="bf16", H=2048, bias=0, mask=True),
        # the full verify batch of 8 drafts, long histories, grammars
        adjust("adjust the full batch", B=512, P=9, V=128256, dtype="bf16", H=8192, bias=64,
               mask=True),
        # plain decoding of one short conversation: latency
        attend("attend one token of one request", B=1, P=1, Hq=32, Hkv=8, D=128, lo=777, hi=777,
               page=16, order="token", dtype="bf16"),
        # plain decoding of a batch of mixed conversations
        attend("attend one token of a batch", B=64, P=1, Hq=32, Hkv=8, D=128, lo=200, hi=8192,
               page=64, order="head", dtype="bf16"),
        # verify of 5 drafts with wide groups: 48 query rows share each key
        attend("attend five drafts of a batch", B=32, P=6, Hq=64, Hkv=8, D=128, lo=500, hi=16384,
               page=32, order="token", dtype="fp16"),
        # verify of 8 drafts over two very long documents, a bias by distance
        attend("attend eight drafts over long caches", B=2, P=9, Hq=32, Hkv=8, D=128, lo=100001,
               hi=131072, page=128, order="token", dtype="bf16", slopes=True),
        # capped scores, a window, wide heads
        attend("attend capped scores in a window", B=16, P=5, Hq=16, Hkv=8, D=256, lo=100,
               hi=8192, page=16, order="head", dtype="bf16", softcap=50.0, window=4096),
        # weights of one verified step of one request
        weigh("weigh one request", B=1, P=5, Hq=32, Hkv=8, D=128, lo=1501, hi=1501, page=16,
              order="token", dtype="bf16"),
        # weights of one verified step of a batch
        weigh("weigh a batch", B=64, P=6, Hq=32, Hkv=8, D=128, lo=1000, hi=8192, page=64,
              order="head", dtype="bf16"),
        # one conversation passes its budget
        evict("evict from one cache", B=1, Hkv=8, D=128, lo=5003, hi=5003, page=16, order="token",
              dtype="bf16", budget=1024, recent=128),
        # a batch of long conversations is cut back, those within the budget move as they are
        evict("evict from a batch", B=64, Hkv=8, D=128, lo=1000, hi=16384, page=64, order="head",
              dtype="fp16", budget=2048, recent=256),
    ]


def adjust(name, *, B, P, V, dtype, H, bias, mask, ragged=1):
    return dict(name=name, op="adjust", B=B, P=P, V=V, dtype=dtype, H=H, bias=bias, mask=mask,
                ragged=ragged)


def attend(name, *, B, P, Hq, Hkv, D, lo, hi, page, order, dtype, softcap=0.0, window=0,
           slopes=False, ragged=1, op="attend"):
    return dict(name=name, op=op, B=B, P=P, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, page=page,
                order=order, dtype=dtype, softcap=softcap, window=window, slopes=slopes,
                ragged=ragged)


def weigh(name, **kw):
    return attend(name, op="weigh", **kw)


def evict(name, *, B, Hkv, D, lo, hi, page, order, dtype, budget, recent, ragged=1):
    return dict(name=name, op="evict", B=B, Hkv=Hkv, D=D, lo=lo, hi=hi, page=page, order=order,
                dtype=dtype, budget=budget, recent=recent, ragged=ragged)


def draw(rng):
    most = {}
    for case in listed():
        w = work(case)
        top = most.setdefault(case["op"], {"bytes": 0.0, "flops": 0.0})
        top.update({k: max(top[k], w[k]) for k in top})
    op = rng.choice(["adjust", "attend", "attend", "weigh", "evict"])
    while True:
        case = _draw(rng, op)
        w = work(case)
        if all(w[k] <= most[op][k] for k in w):
            del case["name"]
            return case


def _draw(rng, op):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    ragged = rng.randrange(1, 1 << 30)
    if op == "adjust":
        return adjust("", B=log(1, 512), P=rng.randint(1, 9), V=log(1000, 152000),
                      dtype=rng.choice(["fp32", "bf16"]), H=log(1, 16384),
                      bias=rng.choice([0, 1, log(1, 300)]), mask=rng.random() < 0.6, ragged=ragged)
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    order = rng.choice(["token", "head"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "evict":
        hi = log(64, 32768)
        budget = max(1, int(hi * rng.uniform(0.05, 0.8)))
        return evict("", B=log(1, 64), Hkv=Hkv, D=D, lo=max(1, hi // rng.randint(1, 20)), hi=hi,
                     page=page, order=order, dtype=dtype, budget=budget,
                     recent=int(budget * rng.random() * 0.6), ragged=ragged)
    make = attend if op == "attend" else weigh
    hi = log(64, 131072)
    return make("", B=log(1, 64), P=rng.randint(1, 9), Hq=Hkv * rng.choice([1, 2, 3, 4, 4, 7, 8]),
                Hkv=Hkv, D=D, lo=max(9, hi // rng.randint(1, 30)), hi=hi, page=page, order=order,
                dtype=dtype, softcap=rng.choice([0.0, 0.0, 30.0]),
                window=rng.choice([0, 0, 0, 500, 4096]), slopes=rng.random() < 0.25, ragged=ragged)


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


def histories(case):
    """(prompt's length, length) of each request's tokens."""
    r = random.Random(case["ragged"] + 2)
    n = [int(round(case["H"] * r.uniform(0.3, 1.0))) for _ in range(case["B"])]
    return [(int(x * r.random()), x) for x in n]


def accepted(case):
    r = random.Random(case["ragged"] + 3)
    return [r.randint(0, n) for n in drafts(case)]


def seen(case, b, n, draft):
    """(first key any row of request b sees, (row, key) pairs seen) of one query head."""
    pos = [n - 1 - draft + i for i in range(draft + 1)]
    start = [max(0, p - case["window"] + 1) if case["window"] else 0 for p in pos]
    return min(start), sum(p + 1 - s for p, s in zip(pos, start))


def work(case):
    B = case["B"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "adjust":
        rows = B + sum(drafts(case))
        read = rows * (case["V"] * size + (4 * -(-case["V"] // 32) if case["mask"] else 0))
        read += sum(4 * n for _, n in histories(case)) + B * (8 * case["bias"] + 4 * case["P"] + 24)
        return {"bytes": float(read + rows * case["V"] * size), "flops": float(2 * rows * case["V"])}
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "evict":
        moved = sum(min(n, case["budget"]) for n in lengths(case))
        return {"bytes": float(sum(4 * n for n in lengths(case)) * Hkv
                               + moved * Hkv * (4 * D * size + 4) + B * Hkv * case["budget"] * 4),
                "flops": float(sum(lengths(case)) * Hkv)}
    G = case["Hq"] // Hkv
    keys = pairs = 0
    acc = accepted(case)
    rows = 0
    for b, (n, d) in enumerate(zip(lengths(case), drafts(case))):
        first, p = seen(case, b, n, d)
        if case["op"] == "weigh":  # the rows up to the last accepted draft
            pos = [n - 1 - d + i for i in range(acc[b] + 1)]
            start = [max(0, x - case["window"] + 1) if case["window"] else 0 for x in pos]
            first, p = min(start), sum(x + 1 - s for x, s in zip(pos, start))
            n = pos[-1] + 1
        keys += n - first
        pairs += p
        rows += d + 1 if case["op"] == "attend" else acc[b] + 1
    if case["op"] == "weigh":
        return {"bytes": float(keys * Hkv * (D * size + 8) + rows * case["Hq"] * (D * size + 4)),
                "flops": float(2 * D * pairs * Hkv * G)}
    return {"bytes": float(keys * Hkv * 2 * D * size + rows * case["Hq"] * (2 * D * size + 4)),
            "flops": float(4 * D * pairs * Hkv * G)}


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    if case["op"] == "adjust":
        return _prepare_adjust(case, g)
    s = _prepare_cache(case, g)
    if case["op"] == "evict":
        return _prepare_evict(case, g, s)
    B, P, Hq, Hkv, D = (case[x] for x in ("B", "P", "Hq", "Hkv", "D"))
    # the queries are a slice of the projection's rows, which hold keys and values too
    qkv = torch.randn((B, P, (Hq + 2 * Hkv) * D), generator=g, device="cuda",
                      dtype=TYPES[case["dtype"]])
    s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
    s["num_draft"] = _ints(drafts(case)) if P > 1 else None
    s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)
                   if case["slopes"] else None)
    s["scale"] = D ** -0.5
    s["out"] = torch.zeros((B, P, Hq, D), dtype=qkv.dtype, device="cuda")
    s["lse"] = torch.zeros((B, P, Hq), dtype=torch.float32, device="cuda")
    if case["op"] == "weigh":
        s["lse"] = _plain_attend(s, case)[1].clone()
        s["accept_len"] = _ints(accepted(case))
        s["prior"] = torch.rand((B, Hkv, case["hi"]), generator=g, device="cuda").square()
        s["weights"] = torch.zeros_like(s["prior"])
    return s


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pool(pages, case, g):
    """A pool of pages [pages, page, Hkv, D] in one of the two orders it is kept in."""
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    shape = (pages, page, Hkv, D) if case["order"] == "token" else (pages, Hkv, page, D)
    t = torch.zeros(shape, device="cuda", dtype=TYPES[case["dtype"]])
    if g is not None:
        t.normal_(generator=g)
    return t if case["order"] == "token" else t.transpose(1, 2)


def _table(counts, width, g):
    """A page table [B, width]: counts[b] pages each, scattered over the pool, then -1."""
    total = sum(counts)
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    have = _ints(counts)[:, None].long()
    first = have.cumsum(0) - have
    at = (first + col).clamp(max=total - 1)
    return torch.where(col < have, ids[at], torch.full_like(ids[at], -1))


def _prepare_cache(case, g):
    n, page = lengths(case), case["page"]
    counts = [-(-x // page) for x in n]
    return {"case": case, "k": _pool(sum(counts), case, g), "v": _pool(sum(counts), case, g),
            "table": _table(counts, max(counts), g), "seq_len": _ints(n)}


def _prepare_evict(case, g, s):
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    # accumulated weights: a few heavy keys, a long light tail, keys nothing ever looked at
    w = torch.empty((B, Hkv, case["hi"]), device="cuda").exponential_(generator=g)
    w = w.pow_(3) * (torch.rand(w.shape, generator=g, device="cuda") < 0.8)
    s["weights"] = w
    counts = [-(-min(x, case["budget"]) // page) for x in lengths(case)]
    s["new_table"] = _table(counts, -(-case["budget"] // page), g)
    s["new_k"] = _pool(sum(counts), case, None)
    s["new_v"] = _pool(sum(counts), case, None)
    return s


def _prepare_adjust(case, g):
    B, P, V, H = case["B"], case["P"], case["V"], case["H"]
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
    # tokens of text repeat: their ranks fall off as a power
    token = lambda *shape: ((V ** rand(*shape) - 1) * 0.999).long().clamp(0, V - 1).to(torch.int32)  # noqa: E731
    s = {"case": case, "logits": torch.randn((B, P, V), generator=g, device="cuda",
                                             dtype=TYPES[case["dtype"]]) * 3}
    s["history"] = token(B, H)
    s["prompt_len"] = _ints([p for p, _ in histories(case)])
    s["hist_len"] = _ints([n for _, n in histories(case)])
    s["draft"] = token(B, P - 1) if P > 1 else None
    s["num_draft"] = _ints(drafts(case)) if P > 1 else None
    s["repetition"] = 1 + 0.3 * rand(B)
    s["presence"] = rand(B) - 0.2
    s["frequency"] = 0.5 * rand(B)
    s["bias_tokens"] = s["bias_values"] = s["allowed"] = None
    if case["bias"]:
        first = torch.randint(0, V, (B, 1), generator=g, device="cuda")
        step = max(1, V // (case["bias"] + 1))
        s["bias_tokens"] = ((first + step * torch.arange(case["bias"], device="cuda")) % V).int()
        s["bias_values"] = 20 * rand(B, case["bias"]) - 10
    if case["mask"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (2, B, P, -(-V // 32)), generator=g, device="cuda",
                              dtype=torch.int64).to(torch.int32)
        # half of the requests are free, the others may emit a quarter of the vocabulary
        free = rand(B, 1, 1) < 0.5
        s["allowed"] = torch.where(free, torch.full_like(words[0], -1), words[0] & words[1])
    s["out"] = torch.zeros((B, P, V), dtype=TYPES[case["dtype"]], device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state, state["case"])
    return _PLAIN[op](state, state["case"])


def _own_adjust(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    return sv.logit_adjust(
        s["logits"], s["history"], s["hist_len"], prompt_len=s["prompt_len"],
        draft_tokens=s["draft"], num_draft=s["num_draft"], repetition=s["repetition"],
        presence=s["presence"], frequency=s["frequency"], bias_tokens=s["bias_tokens"],
        bias_values=s["bias_values"], allowed=s["allowed"], out=s["out"])


def _own_attend(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    return sv.paged_attention(
        s["q"], s["k"], s["v"], s["table"], s["seq_len"], num_draft=s["num_draft"],
        scale=s["scale"], softcap=case["softcap"], window=case["window"], slopes=s["slopes"],
        out=s["out"], out_lse=s["lse"])


def _own_weigh(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    return sv.attention_weight_sum(
        s["q"], s["k"], s["table"], s["seq_len"], s["lse"], num_draft=s["num_draft"],
        accept_len=s["accept_len"], scale=s["scale"], softcap=case["softcap"],
        window=case["window"], slopes=s["slopes"], prior=s["prior"], out=s["weights"])


def _own_evict(s, case):
    import speculative_decoding_verification_17_gb300 as sv

    length, index, weights = sv.kv_cache_evict(
        s["k"], s["v"], s["table"], s["seq_len"], s["weights"], case["budget"], case["recent"],
        s["new_k"], s["new_v"], s["new_table"])
    return length, index, weights, s["new_k"], s["new_v"]


def _plain_adjust(s, case):
    B, P, V, H = case["B"], case["P"], case["V"], case["H"]
    dev = s["logits"].device
    at = torch.arange(H, device=dev)
    inside = at < s["hist_len"][:, None]
    output = inside & (at >= s["prompt_len"][:, None])
    token = s["history"].long()
    any_of = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, token, inside.int())
    out_of = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, token, output.int())
    prefix = torch.zeros((B, P, V), dtype=torch.int32, device=dev)
    if P > 1:
        before = torch.arange(P - 1, device=dev) < torch.arange(P, device=dev)[:, None]
        prefix.scatter_add_(2, s["draft"].long()[:, None].expand(B, P, P - 1).contiguous(),
                            before.int().expand(B, P, P - 1).contiguous())
    z = s["logits"].float()
    factor = s["repetition"][:, None, None]
    z = torch.where(any_of[:, None] + prefix > 0, torch.where(z > 0, z / factor, z * factor), z)
    count = (out_of[:, None] + prefix).float()
    del prefix
    z = z - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    del count
    if s["bias_tokens"] is not None:
        z = z + torch.zeros((B, V), device=dev).scatter_(
            1, s["bias_tokens"].long(), s["bias_values"])[:, None]
    if s["allowed"] is not None:
        bit = torch.arange(V, device=dev, dtype=torch.int32)
        ok = (s["allowed"][:, :, (bit >> 5).long()] >> (bit & 31)) & 1
        z = torch.where(ok.bool(), z, torch.full_like(z, -math.inf))
    if s["num_draft"] is None:
        return z.to(s["out"].dtype)
    live = torch.arange(P, device=dev) <= s["num_draft"][:, None]
    return torch.where(live[..., None], z.to(s["out"].dtype), s["out"])


def _gathered(pool, table, n):
    """The pages of each request in a row: [B, Hkv, n, D] in 32 bits."""
    t = pool[table.clamp(min=0).long()]  # [B, pages, page, Hkv, D]
    return t.flatten(1, 2)[:, :n].transpose(1, 2).float()


def _scores(s, case):
    """(scores [B, Hkv, G, P, n] with what a row does not see at -inf, live rows [B, P])."""
    B, P, Hq, Hkv, n = case["B"], case["P"], case["Hq"], case["Hkv"], case["hi"]
    G = Hq // Hkv
    q = s["q"].float().transpose(1, 2).reshape(B, Hkv, G * P, case["D"])
    z = torch.matmul(q, _gathered(s["k"], s["table"], n).transpose(2, 3)).mul_(s["scale"])
    z = z.view(B, Hkv, G, P, n)
    if case["softcap"]:
        z = torch.tanh(z / case["softcap"]) * case["softcap"]
    row = torch.arange(P, device="cuda")
    draft = (s["num_draft"] if s["num_draft"] is not None else torch.zeros_like(s["seq_len"]))[:, None]
    pos = (s["seq_len"][:, None] - 1 - draft + row)[:, None, None, :, None]
    key = torch.arange(n, device="cuda")
    if s["slopes"] is not None:
        z = z - s["slopes"].view(1, Hkv, G, 1, 1) * (pos - key)
    sees = (key <= pos) & (row <= draft)[:, None, None, :, None]
    if case["window"]:
        sees = sees & (key > pos - case["window"])
    return torch.where(sees, z, torch.full((), -math.inf, device="cuda")), row <= draft


def _plain_attend(s, case):
    B, P, Hq, Hkv, D, n = (case[x] for x in ("B", "P", "Hq", "Hkv", "D", "hi"))
    z, live = _scores(s, case)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z = (z - top).exp_()
    total = z.sum(-1, keepdim=True)
    v = _gathered(s["v"], s["table"], n)
    o = torch.matmul(z.view(B, Hkv, -1, n), v).view(B, Hkv, Hq // Hkv, P, D) / total
    o = o.reshape(B, Hq, P, D).transpose(1, 2).to(s["out"].dtype)
    lse = (top + total.log()).reshape(B, Hq, P).transpose(1, 2)
    return (torch.where(live[..., None, None], o, s["out"]),
            torch.where(live[..., None], lse, s["lse"]))


def _plain_weigh(s, case):
    B, P, Hkv, n = case["B"], case["P"], case["Hkv"], case["hi"]
    z, _ = _scores(s, case)
    lse = s["lse"].transpose(1, 2).reshape(B, Hkv, -1, P, 1)
    counts = torch.arange(P, device="cuda") <= s["accept_len"][:, None]
    p = torch.where(counts[:, None, None, :, None], (z - lse).exp_(), torch.zeros((), device="cuda"))
    inside = torch.arange(n, device="cuda") < s["seq_len"][:, None, None]
    return torch.where(inside, s["prior"] + p.sum((2, 3)), s["weights"])


def _plain_evict(s, case):
    B, Hkv, n, page = case["B"], case["Hkv"], case["hi"], case["page"]
    budget, recent = case["budget"], case["recent"]
    have = s["seq_len"].long()[:, None, None]
    at = torch.arange(n, device="cuda").expand(B, Hkv, n)
    # the last `recent` first, then by weight, what is past the end last; equals by position
    rank = torch.where(at >= have - recent, torch.full((), math.inf, device="cuda"), s["weights"])
    rank = torch.where(at < have, rank, torch.full((), -math.inf, device="cuda"))
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    width = first.shape[-1]
    length = s["seq_len"].clamp(max=budget)
    kept = torch.arange(width, device="cuda") < length[:, None, None]
    index = torch.where(kept, first, torch.full((), n, device="cuda")).sort(-1).values
    at = index.clamp(max=n - 1)
    weights = torch.where(kept, s["weights"].gather(2, at), torch.zeros((), device="cuda"))
    request = torch.arange(B, device="cuda")[:, None, None]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    source = s["table"].long()[request, at // page], at % page, head
    slot = torch.arange(width, device="cuda").expand(B, Hkv, width)
    target = torch.where(kept, s["new_table"].long()[request, slot // page], -1)
    target = target * page + slot % page
    pools = []
    for old, new in ((s["k"], s["new_k"]), (s["v"], s["new_v"])):
        # slots past a request's length land in a row of their own, which is cut off again
        flat = torch.cat([new.reshape(-1, Hkv, case["D"]), new.new_zeros((1, Hkv, case["D"]))])
        flat[torch.where(kept, target, flat.shape[0] - 1), head] = old[source]
        pools.append(flat[:-1].view(new.shape))
    index = torch.where(kept, index, -1).int()
    pad = budget - width
    return (length, torch.nn.functional.pad(index, (0, pad), value=-1),
            torch.nn.functional.pad(weights, (0, pad)), pools[0], pools[1])


_OWN = {"adjust": _own_adjust, "attend": _own_attend, "weigh": _own_weigh, "evict": _own_evict}
_PLAIN = {"adjust": _plain_adjust, "attend": _plain_attend, "weigh": _plain_weigh,
          "evict": _plain_evict}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions, request by request, in 64 bits."""
    s = prepare(case, seed)
    return {"adjust": _exact_adjust, "attend": _exact_attend, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](s, case)


def _exact_adjust(s, case):
    V, P = case["V"], case["P"]
    if case["B"] * P * V > 7e8:
        return None
    out = s["out"].double()
    bits = torch.arange(32, device="cuda", dtype=torch.int32)
    for b, ((prompt, n), d) in enumerate(zip(histories(case), drafts(case))):
        met = torch.bincount(s["history"][b, :n].long(), minlength=V)
        count = torch.bincount(s["history"][b, prompt:n].long(), minlength=V)
        rho, pi, f = (float(s[x][b]) for x in ("repetition", "presence", "frequency"))
        for i in range(d + 1):
            if i:
                met[s["draft"][b, i - 1].long()] += 1
                count[s["draft"][b, i - 1].long()] += 1
            z = s["logits"][b, i].double()
            y = z.clone()
            y[(met > 0) & (z > 0)] /= rho
            y[(met > 0) & (z <= 0)] *= rho
            y -= f * count.double() + pi * (count > 0).double()
            if case["bias"]:
                y[s["bias_tokens"][b].long()] += s["bias_values"][b].double()
            if case["mask"]:
                ok = ((s["allowed"][b, i][:, None] >> bits) & 1).bool().flatten()[:V]
                y[~ok] = -math.inf
            out[b, i] = y
    return out


def _cache_row(s, case, which, b, n):
    page = case["page"]
    ids = s["table"][b, :-(-n // page)].long()
    return s[which][ids].flatten(0, 1)[:n].double()  # [n, Hkv, D]


def _exact_row(s, case, b, n, d):
    """Scores [Hkv, G, d + 1, n] of request b's live rows, -inf where a row does not see."""
    Hkv, D = case["Hkv"], case["D"]
    k = _cache_row(s, case, "k", b, n)
    q = s["q"][b, :d + 1].double().unflatten(1, (Hkv, -1))  # [rows, Hkv, G, D]
    z = torch.einsum("ihgd,jhd->hgij", q, k) / math.sqrt(D)
    if case["softcap"]:
        z = case["softcap"] * torch.tanh(z / case["softcap"])
    away = (n - 1 - d + torch.arange(d + 1, device="cuda"))[:, None] - torch.arange(n, device="cuda")
    if case["slopes"]:
        z -= s["slopes"].double().view(Hkv, -1, 1, 1) * away
    hidden = away < 0
    if case["window"]:
        hidden |= away >= case["window"]
    return z.masked_fill(hidden, -math.inf)


def _exact_attend(s, case):
    out, lse = s["out"].double(), s["lse"].double()
    for b, (n, d) in enumerate(zip(lengths(case), drafts(case))):
        z = _exact_row(s, case, b, n, d)
        total = torch.logsumexp(z, -1)
        p = torch.exp(z - total[..., None])
        o = torch.einsum("hgij,jhd->ihgd", p, _cache_row(s, case, "v", b, n))
        out[b, :d + 1] = o.flatten(1, 2)
        lse[b, :d + 1] = total.flatten(0, 1).transpose(0, 1)
    return out, lse


def _exact_weigh(s, case):
    out = s["weights"].double()
    for b, (n, d) in enumerate(zip(lengths(case), drafts(case))):
        a = accepted(case)[b]
        z = _exact_row(s, case, b, n, d)[:, :, :a + 1]
        lse = s["lse"][b, :a + 1].double().transpose(0, 1).unflatten(0, (case["Hkv"], -1))
        out[b, :, :n] = s["prior"][b, :, :n].double() + torch.exp(z - lse[..., None]).sum((1, 2))
    return out


def _exact_evict(s, case):
    Hkv, page, budget, recent = (case[x] for x in ("Hkv", "page", "budget", "recent"))
    index = torch.full((case["B"], Hkv, budget), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros((case["B"], Hkv, budget), dtype=torch.float64, device="cuda")
    new_k, new_v = s["new_k"].clone(), s["new_v"].clone()
    kept = [min(n, budget) for n in lengths(case)]
    for b, n in enumerate(lengths(case)):
        k, v = (_cache_row(s, case, x, b, n).to(s["k"].dtype) for x in ("k", "v"))
        where = torch.arange(kept[b], device="cuda")
        to = s["new_table"][b].long()[where // page]
        for h in range(Hkv):
            w = s["weights"][b, h, :n]
            if n <= budget:
                keep = where
            else:
                old = n - recent
                heavy = torch.argsort(-w[:old].double(), stable=True)[:budget - recent]
                keep = torch.cat([heavy, torch.arange(old, n, device="cuda")]).sort().values
            index[b, h, :kept[b]] = keep.int()
            weights[b, h, :kept[b]] = w[keep].double()
            new_k[to, where % page, h] = k[keep, h]
            new_v[to, where % page, h] = v[keep, h]
    return _ints(kept), index, weights, new_k.double(), new_v.double()
