"""kv_page_map of a batch without requests."""
import pytest
import torch

import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("P,rows", [(4, None), (None, 0), (None, 1), (None, 700)])
@pytest.mark.parametrize("state", [(3, 5), (0, 9), (8, 0)])
def test_an_empty_batch_keeps_the_ring(P, rows, state):
    ring = i32(list(range(9)))
    args = (torch.empty((0, 6), dtype=torch.int32, device="cuda"), *(i32([]) for _ in range(3)), ring,
            i32(state), 16, 9)
    kw = dict(P=P) if P else dict(rows=rows)

    def same(got):
        torch.cuda.synchronize()
        slots, pos, length, first, new = got
        assert slots.shape == pos.shape == ((0, P) if P else (rows,)) and length.shape == (0,)
        assert bool((slots == -1).all()) and bool((pos == -1).all())
        assert first.tolist() == [0] and new.tolist() == list(state) and ring.tolist() == list(range(9))

    size = (0, P) if P else (rows,)
    made = dict(out_slots=torch.full(size, 7, device="cuda"),
                out_positions=torch.full(size, 7, dtype=torch.int32, device="cuda"), out_len=i32([]),
                out_first=i32([7]), out_state=i32([7, 7]))
    same(sv.kv_page_map(*args, **made))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    same(sv.kv_page_map(*args, **kw, stream=st))
    for t in made.values():
        t.fill_(7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.kv_page_map(*args, **made)
    g.replay()
    same(got)


def test_an_empty_batch_over_a_bad_ring():
    for state in ([-1, 3], [9, 3], [0, 10]):
        none = torch.empty((0, 6), dtype=torch.int32, device="cuda")
        got = sv.kv_page_map(none, *(i32([]) for _ in range(3)), i32(list(range(9))), i32(state), 16, 9, rows=3)
        torch.cuda.synchronize()
        assert got[4].tolist() == [-1, -1] and got[0].tolist() == [-1] * 3


def test_an_idle_step_between_two_others():
    """The ring's state goes from call to call: no page is given out twice."""
    ring, state = i32(list(range(12))), i32([0, 12])
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    _, _, _, _, state = sv.kv_page_map(table, i32([0, 0]), i32([40, 20]), i32([40, 20]), ring, state, 16, 12,
                                       rows=60)
    junk = torch.full((64,), 123456, dtype=torch.int32, device="cuda")  # what freed memory may hold
    del junk
    _, _, _, _, state = sv.kv_page_map(table[:0], i32([]), i32([]), i32([]), ring, state, 16, 12, P=4)
    sv.kv_page_map(table, i32([40, 20]), i32([60, 40]), i32([20, 20]), ring, state, 16, 12, rows=40)
    torch.cuda.synchronize()
    held = [x for x in table.flatten().tolist() if x >= 0]
    assert sorted(held) == list(range(7))
