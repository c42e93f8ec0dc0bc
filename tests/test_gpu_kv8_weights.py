"""The roundings of paged_attention_q8's weights, next to a border."""
import math

import pytest
import torch

import kv8_reference as ref8
import speculative_decoding_verification_17_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [0.1, 0.3, 0.9, 3.1, 5.45, 8.1, 8.7])
def test_weights_are_rounded_to_the_nearest(at):
    """One key takes the row, with a value of 0; 127 others weigh 2^-17 (1 + at / 1024) of it each, which
    fp16 holds to a half step of 2^-28 of the large one's (2^-11 of their own)."""
    cache = ref8.Cache8([128], 64, 64, 1, 64, seed=1, spread=0.0)
    k, v = cache.codes
    k.zero_()
    k[..., 0] = -1.0
    v.fill_(2.0)
    last = int(cache.table[0, 1])
    k[last, 63], v[last, 63] = 0.0, 0.0
    for s in cache.scales:
        s.fill_(1.0)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.float16)
    q[..., 0] = 1.0
    w = 2.0 ** -17 * (1 + at / 1024)
    out, _ = sv.paged_attention_q8(q.cuda(), k.cuda(), v.cuda(), cache.scales[0].cuda(), cache.scales[1].cuda(),
                                   cache.table.cuda(), cache.seq_len.cuda(), scale=-math.log(w))
    want = 127 * w * 2.0 / (1 + 127 * w)
    # the weights' half step, fp16's own of the output, and what the exponent's product is off by: a
    # score of 12 in fp32 through two products and a sum (12 * 3 * 2^-24), the exponential 2^-22
    step = 2.0 ** (math.floor(math.log2(want)) - 10)
    tol = want * 2.0 ** -11 + step / 2 + want * (36 * 2.0 ** -24 + 2.0 ** -21)
    assert bool(((out.cpu()[0, 0, :, 0].double() - want).abs() <= tol).all()), (out[0, 0, 0, 0].item(), want, tol)
