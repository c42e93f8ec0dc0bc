"""The step over a cache in 8 bits as a server runs it: one graph replayed for every step, several
host threads with a stream each, pools past 32 bits of offsets."""
import random
import threading

import pytest
import torch

import kv8_reference as ref8
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class World:
    """A cache and the arrays of a batch's step, all kept in place."""

    def __init__(self, B, P, Hq, Hkv, D, page, block, cols, total, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.P, self.page, self.total = P, page, total
        self.codes = [torch.zeros((total, page, Hkv, D), dtype=ref8.CODE, device="cuda") for _ in range(2)]
        self.scales = [torch.ones((total, page // block, Hkv), device="cuda") for _ in range(2)]
        self.table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        self.ring, self.state = i32(list(range(total))), i32([0, total])
        self.held, self.lens, self.add, self.drafts = (i32([0] * B) for _ in range(4))
        self.freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.x = [torch.zeros((B, P, H, D), dtype=dtype, device="cuda") for H in (Hq, Hkv, Hkv)]
        self.g = g

    def feed(self, held, lens, add):
        for t, v in ((self.held, held), (self.lens, lens), (self.add, add), (self.drafts, [a - 1 for a in add])):
            t.copy_(torch.tensor(v).int())
        for t in self.x:
            t.normal_(generator=self.g)

    def step(self, stream=None):
        """Everything of a step; returns (out, lse, the lengths given)."""
        slots, pos, length, _, state = sv.kv_page_map(self.table, self.held, self.lens, self.add, self.ring,
                                                      self.state, self.page, self.total, P=self.P, stream=stream)
        q, k = sv.qk_norm_rotate(*self.x[:2], pos, self.freq, stream=stream)
        sv.kv_cache_append_q8(k, self.x[2], slots, *self.codes, *self.scales, stream=stream)
        out, lse = sv.paged_attention_q8(q, *self.codes, *self.scales, self.table, length,
                                         num_draft=self.drafts, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.state.copy_(state)
        return out, lse, length


def lengths(B, P, steps, seed):
    """(held, lens, add) of every step: drafts rejected, requests ended and begun."""
    r, held, kept = random.Random(seed), [0] * B, [0] * B
    for _ in range(steps):
        kept = [0 if r.random() < 0.1 else k for k in kept]
        add = [r.randint(1, P) for _ in range(B)]
        lens = [k + a for k, a in zip(kept, add)]
        yield held, lens, add
        held, kept = lens, [n - r.randint(0, a - 1) for n, a in zip(lens, add)]


SHAPE = dict(B=6, P=5, Hq=16, Hkv=4, D=128, page=16, block=16, cols=12, total=60, dtype=torch.bfloat16)


def live_rows(add):
    return torch.arange(SHAPE["P"])[None, :] < torch.tensor(add)[:, None]


def test_a_step_in_one_graph_equals_the_calls():
    """The same bits, step after step, as the calls one by one over a world of their own; and the graph
    captured while another graph of the same calls lives."""
    worlds = [World(seed=1, **SHAPE) for _ in range(3)]
    graphs = []
    for w in worlds[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = w.step()
        graphs.append((g, outs))
    for held, lens, add in lengths(6, 5, 14, seed=5):
        for w in worlds:
            w.feed(held, lens, add)
        want = worlds[0].step()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        live = live_rows(add)
        for w, (_, got) in zip(worlds[1:], graphs):
            assert got[2].tolist() == lens
            for a, b in zip(want[:2], got[:2]):
                assert torch.equal(a.cpu()[live], b.cpu()[live])
            for a, b in zip((*worlds[0].codes, *worlds[0].scales, worlds[0].table, worlds[0].ring, worlds[0].state),
                            (*w.codes, *w.scales, w.table, w.ring, w.state)):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_threads_with_streams_of_their_own():
    steps = [list(lengths(6, 5, 10, seed=s)) for s in range(4)]

    def run(seed, stream, results):
        try:
            w = World(seed=seed, **SHAPE)
            torch.cuda.synchronize()
            outs = []
            for held, lens, add in steps[seed]:
                with torch.cuda.stream(stream):
                    w.feed(held, lens, add)
                    out, lse, _ = w.step(stream=stream)
                    live = live_rows(add)
                    outs.append((out.cpu()[live], lse.cpu()[live]))
            results[seed] = outs
        except Exception as e:  # noqa: BLE001 - read by the test
            results[seed] = e

    alone, together = {}, {}
    for s in range(4):
        run(s, torch.cuda.Stream(), alone)
    threads = [threading.Thread(target=run, args=(s, torch.cuda.Stream(), together)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for s in range(4):
        assert isinstance(alone[s], list) and isinstance(together[s], list), (alone[s], together[s])
        for a, b in zip(alone[s], together[s]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pools_past_32_bits():
    """Keys and values side by side in one pool of 10 GB, whose last pages lie past 2^32 bytes: what is
    written and read there is what a small pool holds."""
    B, P, Hq, Hkv, D, page = 3, 2, 16, 8, 128, 128
    big, small = 40000, 16
    both = torch.empty((big, 2, page, Hkv, D), dtype=torch.uint8, device="cuda").view(ref8.CODE)
    lens, g = [400, 17, 257], torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn((sum(lens), Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B, P, Hq, D), generator=g, device="cuda").bfloat16()
    results = []
    for total, pools in ((big, [both[:, 0], both[:, 1]]),
                         (small, [torch.empty((small, page, Hkv, D), dtype=torch.uint8, device="cuda").view(ref8.CODE)
                                  for _ in range(2)])):
        scales = [torch.full((total, 2, Hkv), float("nan"), device="cuda") for _ in range(2)]
        ids = [total - 1 - 2 * i for i in range(8)]  # (every other one of the last pages)
        table = torch.full((B, 4), -1, dtype=torch.int32)
        slots, at = [], 0
        for b, n in enumerate(lens):
            mine = ids[at:at + -(-n // page)]
            at += len(mine)
            table[b, :len(mine)] = torch.tensor(mine).int()
            slots += [mine[j // page] * page + j % page for j in range(n)]
        sv.kv_cache_append_q8(k, v, torch.tensor(slots, device="cuda"), *pools, *scales)
        out, lse = sv.paged_attention_q8(q, *pools, *scales, table.cuda(), i32(lens))
        torch.cuda.synchronize()
        results.append((out, lse, *(p[ids[0]].view(torch.uint8).clone() for p in pools)))
    assert max(ids) < small and bool(results[0][0].isfinite().all())
    for a, b in zip(*results):
        assert torch.equal(a, b)
