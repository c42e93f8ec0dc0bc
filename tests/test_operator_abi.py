"""The refusals of logit_adjust and of the key-value calls, on the host (no GPU: every call here
returns before any CUDA call), and of their Python binding."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_17_gb300 as sv
from speculative_decoding_verification_17_gb300 import _native

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails or returns first
ODD = ctypes.c_void_p(0x10001)


def adjust(**kw):
    a = dict(z=FAKE, zr=900, zi=300, dtype=0, h=FAKE, hl=FAKE, pl=None, L=64, x=FAKE, nd=None,
             rep=None, pres=None, freq=None, bt=None, bv=None, nb=0, al=None, B=2, P=3, V=300,
             out=ctypes.c_void_p(0x90000), orq=900, oi=300, st=None)
    a.update(kw)
    return sv.library().logit_adjust(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(L=1 << 30), UNSUPPORTED),
    (dict(B=-1), INVALID), (dict(P=0), INVALID), (dict(V=0), INVALID), (dict(dtype=2), INVALID),
    (dict(P=18, zr=99999, orq=99999), UNSUPPORTED), (dict(z=None), INVALID),
    (dict(out=None), INVALID), (dict(h=None), INVALID), (dict(hl=None), INVALID),
    (dict(h=None, hl=None, L=0, pl=FAKE), INVALID), (dict(L=0), INVALID), (dict(L=-1), INVALID),
    (dict(nb=3), INVALID), (dict(nb=-1), INVALID), (dict(bt=FAKE), INVALID),
    (dict(nb=2, bt=FAKE), INVALID), (dict(zi=299), INVALID), (dict(oi=-300), INVALID),
    (dict(zr=899), INVALID), (dict(orq=10), INVALID), (dict(z=ODD), INVALID),
    (dict(hl=ODD), INVALID), (dict(al=ODD), INVALID), (dict(rep=ODD), INVALID),
    (dict(out=FAKE, oi=304, orq=912), INVALID), (dict(B=0, z=None, out=None), OK),
])
def test_logit_adjust_refusals(kw, status):
    assert adjust(**kw) == status


def shape(**kw):
    s = dict(dtype=1, B=2, P=3, Hq=8, Hkv=2, D=128, page_size=16, num_pages=40, max_pages=10)
    s.update(kw)
    return ctypes.byref(_native.KvShape(*s.values()))


def rule(**kw):
    r = dict(scale=0.1, softcap=0.0, window=0, slopes=None)
    r.update(kw)
    return ctypes.byref(_native.ScoreRule(*r.values()))


def pool(data=0x20000, page=4096, token=256, head=128):
    return ctypes.byref(_native.KvPool(data, page, token, head))


WS = ctypes.c_void_p(0x100000)
SHAPES = [
    (dict(dtype=0), INVALID), (dict(dtype=3), INVALID), (dict(B=-1), INVALID),
    (dict(Hkv=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=0), INVALID),
    (dict(page_size=12), UNSUPPORTED), (dict(page_size=4), UNSUPPORTED),
    (dict(page_size=2048), UNSUPPORTED), (dict(page_size=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 26), UNSUPPORTED), (dict(Hkv=2048, Hq=2048), UNSUPPORTED),
]
QUERY_SHAPES = SHAPES + [
    (dict(P=0), INVALID), (dict(P=18), UNSUPPORTED), (dict(Hq=7), INVALID),
    (dict(Hq=130), UNSUPPORTED),
]
RULES = [dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-1.0), dict(softcap=1e-9),
         dict(softcap=float("nan")), dict(window=-1), dict(slopes=0x10002)]
POOLS = [dict(data=0), dict(data=0x20008), dict(page=0), dict(page=-4096), dict(token=100),
         dict(head=4)]


def attend(s=None, r=None, k=None, v=None, **kw):
    a = dict(q=FAKE, q_req=3 * 1024, q_row=1024, q_head=128)
    b = dict(table=FAKE, lens=FAKE, nd=None, out=FAKE, lse=None, ws=WS, wsb=1 << 30, st=None)
    for key, value in kw.items():
        (a if key in a else b)[key] = value
    return sv.library().paged_attention(shape() if s is None else s, rule() if r is None else r,
                                        *a.values(), pool() if k is None else k,
                                        pool() if v is None else v, *b.values())


def weigh(s=None, r=None, k=None, **kw):
    a = dict(q=FAKE, q_req=3 * 1024, q_row=1024, q_head=128)
    b = dict(table=FAKE, lens=FAKE, nd=None, lse=FAKE, lr=24, li=8, lh=1, acc=None, prior=None,
             out=FAKE, stride=160,
             st=None)
    for key, value in kw.items():
        (a if key in a else b)[key] = value
    return sv.library().attention_weight_sum(shape() if s is None else s,
                                             rule() if r is None else r, *a.values(),
                                             pool() if k is None else k, *b.values())


def evict(s=None, **kw):
    a = dict(k=pool(), v=pool(), table=FAKE, lens=FAKE, w=FAKE, stride=160, budget=40, recent=8,
             nk=pool(), nv=pool(), npages=20, ntable=FAKE, ncols=3, ol=FAKE, oi=FAKE, ow=None,
             st=None)
    a.update(kw)
    return sv.library().kv_cache_evict(shape() if s is None else s, *a.values())


def test_shapes_rules_and_pools_are_checked():
    for kw, status in QUERY_SHAPES:
        assert attend(shape(**kw)) == status, kw
        assert weigh(shape(**kw)) == status, kw
        assert sv.library().paged_attention_workspace(shape(**kw)) == 0, kw
    for kw, status in SHAPES:
        assert evict(shape(**kw)) == status, kw
    for kw in RULES:
        assert attend(r=rule(**kw)) == INVALID, kw
        assert weigh(r=rule(**kw)) == INVALID, kw
    for kw in POOLS:
        assert attend(k=pool(**kw)) == INVALID and attend(v=pool(**kw)) == INVALID, kw
        assert weigh(k=pool(**kw)) == INVALID, kw
        for name in ("k", "v", "nk", "nv"):
            assert evict(**{name: pool(**kw)}) == INVALID, kw
    assert sv.library().paged_attention_workspace(shape()) > 0
    huge = dict(B=4096, Hkv=1024, Hq=1024, page_size=1024, max_pages=1 << 19)
    assert attend(shape(**huge)) == UNSUPPORTED and weigh(shape(**huge)) == UNSUPPORTED


def test_pointers_and_strides_are_checked():
    for name in ("q", "table", "lens", "out"):
        assert attend(**{name: None}) == INVALID and attend(**{name: ODD}) == INVALID
    for name in ("q_req", "q_row", "q_head"):
        assert attend(**{name: -8}) == INVALID and attend(**{name: 4}) == INVALID
        assert weigh(**{name: -8}) == INVALID and weigh(**{name: 4}) == INVALID
    assert attend(nd=ODD) == INVALID and attend(lse=ODD) == INVALID
    assert attend(ws=None) == WORKSPACE and attend(wsb=0) == WORKSPACE
    assert attend(ws=ctypes.c_void_p(0x100010)) == WORKSPACE
    for name in ("q", "table", "lens", "lse", "out"):
        assert weigh(**{name: None}) == INVALID and weigh(**{name: ODD}) == INVALID
    assert weigh(lr=-1) == INVALID and weigh(li=-1) == INVALID and weigh(lh=-1) == INVALID
    assert weigh(prior=ODD) == INVALID and weigh(acc=ODD) == INVALID and weigh(stride=0) == INVALID
    for name in ("table", "lens", "w", "ntable", "ol", "oi"):
        assert evict(**{name: None}) == INVALID and evict(**{name: ODD}) == INVALID
    for kw in (dict(budget=0), dict(budget=49), dict(recent=-1), dict(recent=41), dict(stride=0),
               dict(npages=-1), dict(ncols=0), dict(ow=ODD)):
        assert evict(**kw) == INVALID, kw


def test_no_requests_is_a_no_op():
    none = shape(B=0)
    assert attend(none, q=None, table=None, out=None, ws=None) == OK
    assert weigh(none, q=None, out=None) == OK
    assert evict(none, table=None, ol=None) == OK


def test_binding_refuses_host_tensors():
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    kv = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16)
    table, n = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        sv.paged_attention(q, kv, kv, table, n)
    with pytest.raises(TypeError):
        sv.attention_weight_sum(q, kv, table, n, torch.zeros((1, 1, 2)))
    with pytest.raises(TypeError):
        sv.kv_cache_evict(kv, kv, table, n, torch.zeros((1, 1, 32)), 16, 0, kv, kv, table)
    with pytest.raises(TypeError):
        sv.logit_adjust(torch.zeros((1, 1, 8)))
    with pytest.raises(TypeError):
        sv.logit_adjust(torch.zeros((1, 1, 8), dtype=torch.float16))
