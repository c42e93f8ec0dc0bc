"""Speculative decoding around a paged cache, with every step of it on the device.

A toy one-layer decoder (random weights) generates for a small batch:

  ngram_propose         drafts from what each request has said so far
  paged_attention       the k+1 new positions over the paged key-value cache
  logit_adjust          penalties and a token ban on the rows of all positions
  spec_verify_greedy    keeps the longest prefix the model itself would have said
  attention_weight_sum  what the accepted positions looked at (rejected drafts do not count)
  kv_cache_evict        cuts a cache back to its budget once it has grown past it

Run it on a GPU: ``python examples/verify_step.py``. With ``k = 0`` the same loop decodes token by
token; the drafts change how many steps it takes, not what comes out.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_17_gb300 as sv  # noqa: E402

V, WIDTH, HQ, HKV, D, PAGE = 512, 256, 4, 2, 64, 16


class Toy:
    """Random weights of the toy decoder; positions enter through a per-position rotation of the
    queries and keys, so a key keeps its position wherever its slot moves."""

    def __init__(self, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.embed = rand(V, WIDTH)
        self.qkv = rand(WIDTH, (HQ + 2 * HKV) * D) * WIDTH ** -0.5
        self.mix = rand(HQ * D, WIDTH) * (HQ * D) ** -0.5
        self.head = rand(WIDTH, V) * WIDTH ** -0.5
        self.angle = 10000.0 ** (-torch.arange(D // 2, device=device) / (D // 2))

    def rotate(self, x, pos):
        a = pos[..., None, None].float() * self.angle
        x1, x2 = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([x1 * a.cos() - x2 * a.sin(), x1 * a.sin() + x2 * a.cos()], -1)

    def project(self, tokens, pos):
        """Queries [B, P, HQ, D], keys and values [B, P, HKV, D] of tokens at positions."""
        x = self.embed[tokens.clamp(min=0).long()]
        q, k, v = (x @ self.qkv).unflatten(-1, (HQ + 2 * HKV, D)).split([HQ, HKV, HKV], -2)
        return (x, *(t.to(torch.bfloat16) for t in (self.rotate(q, pos), self.rotate(k, pos), v)))

    def logits(self, x, attended):
        return (x + attended.float().flatten(-2) @ self.mix) @ self.head


def append(pool, new, table, slot, live):
    """Writes new [B, P, HKV, D] into the slots [B, P] of each request's pages, where live."""
    page = table.gather(1, (slot // PAGE).clamp(max=table.shape[1] - 1).long())
    # what is not live goes to the pool's last page, which no request uses
    page = torch.where(live, page, pool.shape[0] - 1).long()
    pool[page, (slot % PAGE).long()] = new


def generate(prompts, steps, k, *, budget=0, recent=16, banned=(), repetition=1.0,
             device="cuda", seed=0):
    """Token lists that continue the prompts by `steps` tokens, and how many steps ran.
    With a budget, caches past it are cut back to it (the heaviest and the most recent keys)."""
    model = Toy(device, seed)
    B, P = len(prompts), k + 1
    longest = max(map(len, prompts)) + steps + 2 * P  # (a last step may say P tokens)
    cols = -(-longest // PAGE)
    i32 = dict(dtype=torch.int32, device=device)
    history = torch.full((B, longest), -1, **i32)
    for b, p in enumerate(prompts):
        history[b, :len(p)] = torch.tensor(p, **i32)
    prompt_len = torch.tensor([len(p) for p in prompts], **i32)
    hist_len = prompt_len.clone()
    # two sets of pages per request: an eviction moves a cache from one to the other
    tables = torch.arange(2 * B * cols, **i32).view(2, B, cols)
    shape = (2 * B * cols + 1, PAGE, HKV, D)
    pool_k, pool_v = (torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2))
    seen = torch.zeros((B, HKV, cols * PAGE), device=device)  # the weight each key received
    cached = torch.zeros(B, **i32)  # slots in use, the newest token's not among them yet
    current = 0
    mask = torch.full((B, P, V // 32), -1, **i32)
    for t in banned:
        mask[..., t // 32] &= ~(1 << (t % 32)) if t % 32 < 31 else 0x7fffffff
    penalty = torch.full((B,), repetition, device=device)
    at = torch.arange(max(P, 1), device=device)

    # the prompts, position by position (a prefill would do them at once)
    for i in range(int(prompt_len.max()) - 1):
        live = (i < prompt_len - 1)[:, None]
        _, _, nk, nv = model.project(history[:, i:i + 1], torch.full((B, 1), i, device=device))
        append(pool_k, nk, tables[0], cached[:, None], live)
        append(pool_v, nv, tables[0], cached[:, None], live)
        cached += live[:, 0].int()

    ran = 0
    while int((hist_len - prompt_len).min()) < steps:
        ran += 1
        active = hist_len - prompt_len < steps  # a request that is done waits for the others
        if k:
            draft, num_draft = sv.ngram_propose(history, hist_len, 3, 1, k)
            num_draft = torch.where(active, num_draft, 0)
        else:
            draft, num_draft = torch.zeros((B, 0), **i32), torch.zeros(B, **i32)
        tokens = torch.cat([history.gather(1, (hist_len - 1)[:, None].long()), draft], 1)
        pos = (hist_len - 1)[:, None] + at[None, :P]
        x, q, nk, nv = model.project(tokens, pos)
        table = tables[current]
        slots, live = cached[:, None] + at[None, :P], at[None, :P] <= num_draft[:, None]
        append(pool_k, nk, table, slots, live)
        append(pool_v, nv, table, slots, live)
        length = cached + 1 + num_draft
        attended, lse = sv.paged_attention(q, pool_k, pool_v, table, length, num_draft=num_draft,
                                           out=torch.zeros_like(q, memory_format=torch.contiguous_format))
        logits = sv.logit_adjust(model.logits(x, attended), history, hist_len,
                                 prompt_len=prompt_len, draft_tokens=draft if k else None,
                                 num_draft=num_draft, repetition=penalty, allowed=mask)
        if k:
            said, accepted = sv.spec_verify_greedy(logits, draft, num_draft)
        else:
            said, accepted = logits.argmax(-1).int(), torch.zeros(B, **i32)
        sv.attention_weight_sum(q, pool_k, table, length, lse, num_draft=num_draft,
                                accept_len=accepted, prior=seen, out=seen)
        # commit: the accepted drafts and the model's own next token
        new = torch.where(active, accepted + 1, 0)
        cols_of = torch.where(at[None, :P] < new[:, None], hist_len[:, None] + at[None, :P],
                              longest - 1)
        history.scatter_(1, cols_of.long(), torch.where(at[None, :P] < new[:, None], said, -1))
        hist_len += new
        cached += new
        if budget and int(cached.max()) > budget:
            keep, _, weights = sv.kv_cache_evict(
                pool_k, pool_v, table, cached, seen, budget, recent, pool_k, pool_v,
                tables[1 - current])
            cached, current = keep, 1 - current
            seen.zero_()
            seen[:, :, :budget] = weights
        else:  # slots of rejected drafts are written again by the next step
            seen.masked_fill_(torch.arange(cols * PAGE, device=device) >= cached[:, None, None], 0)
    out = history.cpu()
    return [out[b, n:n + steps].tolist() for b, n in enumerate(prompt_len.tolist())], ran


def main():
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, V, (n,), generator=g).tolist() * 3 for n in (5, 9, 12, 7)]
    plain, plain_steps = generate(prompts, 60, 0)
    drafted, steps = generate(prompts, 60, 5)
    print(f"token by token: {plain_steps} steps; with 5 drafts: {steps} steps; "
          f"the same tokens: {plain == drafted}")
    cut, _ = generate(prompts, 60, 5, budget=48, banned=(7, 63), repetition=1.2)
    print("repeats penalised, two tokens banned, a cache of 48 keys:", cut[0][:12], "...")


if __name__ == "__main__":
    main()
