"""The operators of a step over a cache in 8 bits, in 64 bits on the CPU from their definitions, with
the error bounds the GPU tests hold the kernels to."""
import math

import torch

from kv_reference import HALF_STEP

CODE = torch.float8_e4m3fn


def code_of(x):
    """The nearest e4m3 value (ties to even) of doubles within its range; NaN stays."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


class Cache8:
    """A paged cache of codes on the CPU: pools of scattered pages whose unused slots hold NaN codes,
    and whose unused blocks have NaN scales."""

    def __init__(self, lens, page, block, Hkv, D, *, order="token", seed=0, spare=3, spread=1.0,
                 plain_scales=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.block, self.D, self.order = list(lens), page, block, D, order
        counts = [-(-n // page) for n in lens]
        total = sum(counts) + spare
        self.max_pages = max(1, max(counts, default=1))
        ids = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        self.codes = [torch.full((total, page, Hkv, D), math.nan, dtype=CODE) for _ in range(2)]
        self.scales = [torch.full((total, page // block, Hkv), math.nan) for _ in range(2)]
        at = 0
        for b, (n, c) in enumerate(zip(lens, counts)):
            mine = ids[at:at + c]
            self.table[b, :c] = mine
            at += c
            for codes, scales in zip(self.codes, self.scales):
                x = torch.randn((c * page, Hkv, D), generator=g)
                size = torch.exp(spread * torch.randn((c * page // block, Hkv), generator=g))
                if plain_scales:
                    size = torch.exp2(torch.round(torch.log2(size)))
                x = (x * 64).clamp(-448, 448).to(CODE)
                x[n:] = math.nan
                size[-(-n // block):] = math.nan
                codes[mine.long()] = x.view(c, page, Hkv, D)
                scales[mine.long()] = size.view(c, page // block, Hkv) / 64
        self.seq_len = torch.tensor(self.lens, dtype=torch.int32)

    def view(self, which, device="cpu"):
        t = self.codes[which]
        if self.order == "head":
            return t.view(torch.uint8).transpose(1, 2).contiguous().view(CODE).to(device).transpose(1, 2)
        return t.to(device)

    def row(self, which, b, h):
        """Keys or values of a request's kv head [n, D], in double."""
        n = self.lens[b]
        at = self.table[b, :-(-n // self.page)].long()
        x = self.codes[which][:, :, h].double()[at].flatten(0, 1)[:n]
        s = self.scales[which][at][:, :, h].double().flatten().repeat_interleave(self.block)[:n]
        return x * s[:, None]


def attention8(cache, q, num_draft, *, scale, softcap=0.0, window=0, slopes=None):
    """(out, lse, bound on out, bound on lse), [B, P, Hq, ...]; rows past num_draft NaN in the bounds."""
    B, P, Hq, D = q.shape
    Hkv = cache.codes[0].shape[2]
    G, half = Hq // Hkv, HALF_STEP[q.dtype]
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.full(q.shape, math.nan, dtype=torch.float64)
    lse = torch.zeros((B, P, Hq), dtype=torch.float64)
    tol_lse = torch.full((B, P, Hq), math.nan, dtype=torch.float64)
    for b in range(B):
        n, rows = cache.lens[b], num_draft[b] + 1
        pos = (n - 1 - num_draft[b] + torch.arange(rows))[:, None, None]
        j = torch.arange(n)
        for h in range(Hkv):
            k, v = cache.row(0, b, h), cache.row(1, b, h)
            at = slice(h * G, (h + 1) * G)
            x = q[b, :rows, at].double()
            s = torch.einsum("pgd,nd->pgn", x, k) * scale
            # the instruction adds up in fp32 and cuts (2^-20.7 of the absolute sum, measured, over
            # 128 products; four times that here), and a query element is off by 2^-17 of its row's
            # largest where it is below 2^-6 of it
            err = abs(scale) * (2.0 ** -18.7 * torch.einsum("pgd,nd->pgn", x.abs(), k.abs())
                                + 2.0 ** -17 * x.abs().amax(-1, keepdim=True) * k.abs().sum(-1))
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                err = err + softcap * 2.0 ** -21
            away = (pos - j).double()
            slope = 0.0 if slopes is None else slopes[at].double()[None, :, None]
            err = err + 2.0 ** -22 * (away.abs() * abs(slope) + s.abs())
            s = s - slope * away
            sees = (j <= pos) & (j > pos - window if window else j >= 0)
            sees = sees.expand(s.shape)
            s = s.masked_fill(~sees, -math.inf)
            live = sees.any(-1)
            l = torch.where(live, torch.logsumexp(s, -1) if n else 0.0, -math.inf)
            p = torch.where(sees, torch.exp(s - torch.where(live, l, 0.0)[..., None]), 0.0)
            o = torch.einsum("pgn,nd->pgd", p, torch.where(torch.isfinite(v), v, 0.0))
            meets = torch.einsum("pgn,nd->pgd", sees.double(), torch.isnan(v).double())
            o = torch.where(meets > 0, math.nan, o)  # a NaN code that the row sees
            size = torch.einsum("pgn,nd->pgd", p, v.abs().nan_to_num(0.0))
            worst = torch.where(sees, err, 0.0).amax(-1) if n else torch.zeros(rows, G)
            # a weight is off by its score's error (twice: it and the sum), the exponential's, the
            # sums' and the rounding to fp16 (2^-11 of it at worst); the accumulator cuts each of its additions
            w = 2 * worst + 2.0 ** -21 + (n + 8) * 2.0 ** -23 + 2.0 ** -11 + (n / 32 + 8) * 2.0 ** -22
            t = w[..., None] * size + half * o.abs() + (2.0 ** -24 if q.dtype == torch.float16 else 1e-30)
            if n:
                # and by 2^-17, half the last step of what weights are cut into, in units in which the
                # largest weight times its scale is 2^10 (bf16) or 2^11 (fp16) or more: 2^-27, 2^-28
                big = (p * (v.abs().amax(-1) / 32).nan_to_num(0.0)).amax(-1)  # (a row of codes reaches 32)
                t = t + (2.0 ** -28 if q.dtype == torch.float16 else 2.0 ** -27) * big[..., None] * 448 * n
            out[b, :rows, at], tol[b, :rows, at] = o, t
            lse[b, :rows, at] = l
            tol_lse[b, :rows, at] = worst + (n + 8) * 2.0 ** -23 + 2.0 ** -21 * (1 + l.abs().nan_to_num(0, 0, 0))
    return out, lse, tol, tol_lse


def need(top):
    """The smallest power of two, 2^-40 at least, that brings a magnitude within 448."""
    return torch.exp2(torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -40))))


def append8(x, slots, codes, scales, block):
    """(codes, scales) in double after new rows x [T, Hkv, D] went to their slots; codes NaN stay.
    Quotients are those of fp32: exact by a power of two, and rounded once more by another scale."""
    codes, scales = codes.double().clone(), scales.double().clone()
    pages, page = codes.shape[:2]
    limit = 448 * 2.0 ** 40
    x = x.double()
    t = 0
    while t < len(slots):
        if not 0 <= slots[t] < pages * page:
            t += 1
            continue
        end = t + 1
        while end < len(slots) and 0 <= slots[end] < pages * page and slots[end] // block == slots[t] // block:
            end += 1
        p, first = slots[t] // page, slots[t] % page
        c = first // block
        rows = x[t:end]
        good = rows.abs() <= limit  # (NaN is not)
        now = need(torch.where(good, rows.abs(), 0.0).amax((0, 2)))
        if any(a >= b for a, b in zip(slots[t:end], slots[t + 1:end])):
            scales[p, c] = math.nan
            t = end
            continue
        if first % block:
            was = scales[p, c]
            bad = ~((was >= 0) & (was <= 2.0 ** 40))
            now = torch.where(bad, math.nan, torch.maximum(now, was))
            old = codes[p, c * block:first]
            ratio = torch.where(bad | (now == was), 1.0, was / now)
            codes[p, c * block:first] = code_of((old.float() * ratio.float()[:, None]).double())
        scales[p, c] = now
        for i in range(t, end):
            codes[p, slots[i] % page] = code_of(
                (torch.where(good[i - t], x[i], math.nan).float() / now.float()[:, None]).double())
        t = end
    return codes, scales


def page_map(table, old_len, seq_len, num_new, ring, state, page, num_pages, P, rows):
    """kv_page_map's definition over lists; returns (slots, positions, out_len, first, state) and
    changes table and ring."""
    size, (head, count) = len(ring), state
    B, most = len(old_len), len(table[0]) * page if table else 0
    up = lambda n: -(-n // page)  # noqa: E731
    first, at, fine = [], 0, []
    for b in range(B):
        a, n, x = old_len[b], seq_len[b], num_new[b]
        ok = 0 <= a <= most and 0 <= n <= most and 0 <= x <= n and (not P or x <= P)
        first.append(b * P if P else at)
        at += x if ok else 0
        fine.append(ok and (P or at <= rows))
    first.append(B * P if P else at)
    slots, positions, out_len = [-1] * rows, [-1] * rows, [-1] * B
    back = sum(max(0, up(old_len[b]) - up(seq_len[b])) for b in range(B) if fine[b])
    if not (0 <= head < size and 0 <= count <= size and count + back <= size):
        return slots, positions, out_len, first, (-1, -1)
    asked = taken = 0
    given = []
    for b in range(B):
        if not fine[b]:
            continue
        have, want = up(old_len[b]), up(seq_len[b])
        asked += max(0, want - have)
        if want > have and asked > count:
            out_len[b] = old_len[b]
            continue
        out_len[b] = seq_len[b]
        for t in range(have, want):
            table[b][t] = ring[(head + taken) % size]
            taken += 1
        given += table[b][want:have]
        for i in range(num_new[b]):
            p = seq_len[b] - num_new[b] + i
            of = table[b][p // page]
            positions[first[b] + i] = p
            if 0 <= of < num_pages:
                slots[first[b] + i] = of * page + p % page
    for i, x in enumerate(given):
        ring[(head + count + i) % size] = x
    return slots, positions, out_len, first, ((head + taken) % size, count - taken + len(given))


def norm_rotate(x, positions, inv_freq, weight, eps, norm, interleaved):
    """(result [T, heads, D], bound) of rows x [T, heads, D]."""
    D = x.shape[-1]
    y = x.double()
    if norm:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    R = 2 * len(inv_freq)
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., :R // 2], y[..., R // 2:R])
    t = positions.double()[:, None] * inv_freq.double()
    c, s = t.cos()[:, None], t.sin()[:, None]
    pair = (a * c - b * s, a * s + b * c)
    turned = torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1)
    out = torch.cat([turned, y[..., R:]], -1)
    mate = torch.hypot(a, b)
    mate = torch.stack([mate, mate], -1).flatten(-2) if interleaved else torch.cat([mate, mate], -1)
    size = torch.cat([mate, y[..., R:].abs()], -1)
    # the angle: 2^-53 of the turns (t / 2 pi) in the frequency, 2^-24 of half a turn when rounded; sine
    # and cosine (2^-23), products and sums (six half steps), the root (2^-21), the output's rounding
    angle = t.abs().amax() * 2.0 ** -51 if R else 0.0
    err = (angle + math.pi * 2.0 ** -24 + 2.0 ** -22 + 6 * 2.0 ** -24 + (D + 8) * 2.0 ** -25 + 2.0 ** -21) * size
    return out, err + HALF_STEP[x.dtype] * out.abs() + (2.0 ** -24 if x.dtype == torch.float16 else 1e-38)
