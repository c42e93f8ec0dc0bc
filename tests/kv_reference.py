"""The paged cache's operators and the logits' adjustment in 64 bits on the CPU, from their
definitions, with the error bounds the GPU tests hold the kernels to."""
import math

import torch

# half a step of a rounding to the type, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Cache:
    """A paged cache on the CPU: pools of scattered pages whose unused slots hold ``fill``."""

    def __init__(self, lens, page, Hkv, D, dtype, *, max_pages=None, order="token", fill=math.nan,
                 seed=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.D = list(lens), page, D
        counts = [-(-n // page) for n in lens]
        total = sum(counts) + spare
        self.max_pages = max_pages or max(1, max(counts))
        ids = torch.randperm(total, generator=g).tolist()
        self.table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
            at += c
        shape = (total, page, Hkv, D) if order == "token" else (total, Hkv, page, D)
        self.pools = []
        for _ in range(2):
            pool = torch.full(shape, fill, dtype=dtype)
            view = pool if order == "token" else pool.transpose(1, 2)
            for b, n in enumerate(self.lens):
                for j in range(n):
                    view[self.table[b, j // page], j % page] = torch.randn(
                        (Hkv, D), generator=g).to(dtype)
            self.pools.append(pool)
        self.order = order
        self.seq_len = torch.tensor(self.lens, dtype=torch.int32)

    def view(self, which, device=None):
        pool = self.pools[which] if device is None else self.pools[which].to(device)
        return pool if self.order == "token" else pool.transpose(1, 2)

    def row(self, which, b, h):
        """Keys or values of a request's kv head [n, D], in double."""
        v = self.view(which)
        return torch.stack([v[self.table[b, j // self.page], j % self.page, h]
                            for j in range(self.lens[b])]).double() if self.lens[b] else \
            torch.zeros((0, self.D), dtype=torch.float64)


def score_row(q, k, pos, *, scale, softcap=0.0, window=0, slope=0.0):
    """(scores of one row [n], which keys it sees, a bound on an fp32 score's error)."""
    n = k.shape[0]
    j = torch.arange(n)
    qk = k @ q
    # D products summed in any order in fp32: at most D half steps of the absolute sum
    err = (q.numel() + 4) * 2.0 ** -24 * abs(scale) * (k.abs() @ q.abs())
    s = qk * scale
    if softcap:
        s = softcap * torch.tanh(s / softcap)
        err = err + softcap * 2.0 ** -21  # tanh from one exponential and one quotient
    away = (pos - j).double()
    err = err + 2.0 ** -22 * (abs(slope) * away.abs() + s.abs())
    s = s - slope * away
    sees = j <= pos
    if window:
        sees &= j > pos - window
    return s, sees, err


def attention(cache, q, num_draft, **rule):
    """For every live row (b, i, head): (out [D], lse, bound on out, bound on lse); the bounds
    hold for scores, weights and sums in fp32 with the weights rounded once to q's type."""
    B, P, Hq, D = q.shape
    Hkv = cache.view(0).shape[2]
    slopes = rule.pop("slopes", None)
    half = HALF_STEP[q.dtype]
    res = {}
    for b in range(B):
        for h in range(Hkv):
            k, v = cache.row(0, b, h), cache.row(1, b, h)
            for i in range(num_draft[b] + 1):
                pos = cache.lens[b] - 1 - num_draft[b] + i
                for head in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    slope = float(slopes[head]) if slopes is not None else 0.0
                    s, sees, err = score_row(q[b, i, head].double(), k, pos, slope=slope, **rule)
                    if not bool(sees.any()):
                        res[b, i, head] = (torch.zeros(D, dtype=torch.float64), -math.inf,
                                           torch.zeros(D, dtype=torch.float64), 0.0)
                        continue
                    s, vv, err = s[sees], v[sees], float(err[sees].max())
                    lse = torch.logsumexp(s, 0)
                    p = torch.exp(s - lse)
                    out = p @ vv
                    # every weight is off by its score's error (twice: it and the sum), the
                    # exponential's (2^-22), the sums' (a half step per term) and one rounding
                    w = 2 * err + 2.0 ** -21 + (s.numel() + 8) * 2.0 ** -23 + half
                    tol = w * (p @ vv.abs()) + half * out.abs() + 1e-30
                    if q.dtype == torch.float16:
                        tol = tol + 2.0 ** -24  # the output's subnormals
                    tol_lse = err + (s.numel() + 8) * 2.0 ** -24 + 2.0 ** -21 * (1 + abs(float(lse)))
                    res[b, i, head] = (out, float(lse), tol, tol_lse)
    return res


def weight_sum(cache, q, num_draft, accept_len, lse, prior, **rule):
    """(sums [B, Hkv, N], their bound) for the slots below each length; prior elsewhere."""
    B, P, Hq, D = q.shape
    Hkv = cache.view(0).shape[2]
    slopes = rule.pop("slopes", None)
    out, tol = prior.double().clone(), torch.zeros_like(prior, dtype=torch.float64)
    for b in range(B):
        n = cache.lens[b]
        for h in range(Hkv):
            k = cache.row(0, b, h)
            for i in range(accept_len[b] + 1):
                pos = n - 1 - num_draft[b] + i
                for head in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    if lse[b, i, head] == -math.inf:
                        continue
                    slope = float(slopes[head]) if slopes is not None else 0.0
                    s, sees, err = score_row(q[b, i, head].double(), k, pos, slope=slope, **rule)
                    w = torch.where(sees, torch.exp(s - lse[b, i, head].double()), 0.0)
                    out[b, h, :n] += w
                    tol[b, h, :n] += w * (err + 2.0 ** -21 + 2.0 ** -22 * lse[b, i, head].abs())
            rows = (accept_len[b] + 2) * (Hq // Hkv)
            tol[b, h, :n] += rows * 2.0 ** -24 * out[b, h, :n].abs()
    return out, tol


def evict(weights, lens, budget, recent):
    """Kept slots of every (request, head), in order; ties to the lowest slot, NaN as -inf."""
    kept = {}
    for b, n in enumerate(lens):
        for h in range(weights.shape[1]):
            if n <= budget:
                kept[b, h] = list(range(n))
                continue
            w = [(-math.inf if math.isnan(x) else x) for x in weights[b, h, :n].tolist()]
            old = sorted(range(n - recent), key=lambda j: (-w[j], j))[:budget - recent]
            kept[b, h] = sorted(old + list(range(n - recent, n)))
    return kept


def adjust(logits, *, history=None, hist_len=None, prompt_len=None, draft=None, num_draft=None,
           repetition=None, presence=None, frequency=None, bias_tokens=None, bias_values=None,
           allowed=None):
    """(adjusted logits [B, P, V] in double, a bound on the kernel's error); rows past num_draft
    are NaN in the bound."""
    B, P, V = logits.shape
    out = logits.double().clone()
    tol = torch.full((B, P, V), math.nan, dtype=torch.float64)
    get = lambda t, b, d: d if t is None else float(t[b])  # noqa: E731
    for b in range(B):
        n = 0 if hist_len is None else int(hist_len[b])
        prompt = 0 if prompt_len is None else int(prompt_len[b])
        nd = P - 1 if num_draft is None else int(num_draft[b])
        rho, pi, f = get(repetition, b, 1.0), get(presence, b, 0.0), get(frequency, b, 0.0)
        bias = {}
        if bias_tokens is not None:
            for t, x in zip(bias_tokens[b].tolist(), bias_values[b].tolist()):
                bias.setdefault(t, x)
        for i in range(nd + 1):
            seen, count = set(), {}
            ahead = [] if draft is None else draft[b, :i].tolist()
            tokens = [] if history is None else history[b, :n].tolist()
            for at, t in list(enumerate(tokens)) + [(math.inf, t) for t in ahead]:
                seen.add(t)
                if at >= prompt:
                    count[t] = count.get(t, 0) + 1
            z = logits[b, i].double()
            y, size = z.clone(), z.abs()
            for t in seen:
                if 0 <= t < V:
                    y[t] = y[t] / rho if y[t] > 0 else y[t] * rho
                    size[t] = torch.maximum(size[t], y[t].abs())
            for t, c in count.items():
                if 0 <= t < V:
                    y[t] -= f * c + pi
                    size[t] += abs(f) * c + abs(pi)
            for t, x in bias.items():
                if 0 <= t < V:
                    y[t] += x
                    size[t] += abs(x)
            if allowed is not None:
                bits = (allowed[b, i][:, None] >> torch.arange(32, dtype=torch.int32)) & 1
                y[~bits.flatten()[:V].bool()] = -math.inf
            out[b, i] = y
            # seven fp32 operations at most on a logit, then the output's rounding
            bound = 8 * 2.0 ** -24 * size + HALF_STEP[logits.dtype] * y.abs()
            tol[b, i] = bound.nan_to_num(0.0, 0.0, 0.0)
    return out, tol


def close(got, want, tol):
    """Whether got is within tol of want everywhere (equal infinities and NaNs included)."""
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    return bool((same | ((got - want).abs() <= tol)).all())


def attention_on_device(q, k, v, table, lens, num_draft, *, scale, softcap=0.0, window=0,
                        slopes=None):
    """paged_attention's definition and bounds for many requests, in 64 bits with the pools (zeros
    past every length) on q's device: (out, lse, bound on out, bound on lse, live rows)."""
    B, P, Hq, D = q.shape
    pages, page, Hkv, _ = k.shape
    n = int(lens.max()) if B else 0
    cols = max(1, -(-n // page))
    row = lambda pool: pool[table[:, :cols].clamp(min=0).long()].flatten(1, 2)[:, :n].double()  # noqa: E731
    kk, vv = row(k), row(v)  # [B, n, Hkv, D]
    qq = q.double().unflatten(2, (Hkv, -1))
    s = torch.einsum("bphgd,bnhd->bhgpn", qq, kk) * scale
    err = (D + 4) * 2.0 ** -24 * abs(scale) * torch.einsum("bphgd,bnhd->bhgpn", qq.abs(), kk.abs())
    if softcap:
        s = softcap * torch.tanh(s / softcap)
        err = err + softcap * 2.0 ** -21
    i, j = torch.arange(P, device=q.device), torch.arange(n, device=q.device)
    pos = (lens[:, None] - 1 - num_draft[:, None] + i)[:, None, None, :, None]
    slope = 0.0 if slopes is None else slopes.double().view(1, Hkv, -1, 1, 1)
    away = (pos - j).double()
    err = err + 2.0 ** -22 * (away.abs() * abs(slope) + s.abs())
    s = s - slope * away
    sees = j <= pos
    if window:
        sees = sees & (j > pos - window)
    s = s.masked_fill(~sees, -math.inf)
    any_key = sees.any(-1, keepdim=True).expand(*s.shape[:-1], 1)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.where(any_key, torch.exp(s - lse), 0.0).nan_to_num(0.0)
    out = torch.einsum("bhgpn,bnhd->bphgd", p, vv).flatten(2, 3)
    size = torch.einsum("bhgpn,bnhd->bphgd", p, vv.abs()).flatten(2, 3)
    worst = torch.where(sees, err, 0.0).amax(-1)  # [B, Hkv, G, P]
    worst = worst.flatten(1, 2).transpose(1, 2)
    half = HALF_STEP[q.dtype]
    w = 2 * worst[..., None] + 2.0 ** -21 + (n + 8) * 2.0 ** -23 + half
    lse = lse[..., 0].flatten(1, 2).transpose(1, 2)
    tol = w * size + half * out.abs() + (2.0 ** -24 if q.dtype == torch.float16 else 1e-30)
    tol_lse = worst + (n + 8) * 2.0 ** -24 + 2.0 ** -21 * (1 + lse.abs().nan_to_num(0, 0, 0))
    return out, lse, tol, tol_lse, i <= num_draft[:, None]
