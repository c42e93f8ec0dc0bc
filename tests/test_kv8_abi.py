"""The refusals of the calls of a step over a cache in 8 bits, on the host (no GPU: every call here
returns before any CUDA call), and of their Python binding."""
import ctypes
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import speculative_decoding_verification_17_gb300 as sv
from speculative_decoding_verification_17_gb300 import _native

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE, ODD = 0x10000, 0x10001


def shape(**kw):
    s = dict(dtype=1, B=2, P=3, Hq=8, Hkv=2, D=128, page_size=16, num_pages=40, max_pages=10)
    s.update(kw)
    return ctypes.byref(_native.KvShape(*s.values()))


def pool(data=0x20000, page=4096, token=256, head=128):
    return ctypes.byref(_native.KvPool(data, page, token, head))


POOLS = [dict(data=None), dict(data=0x20008), dict(page=0), dict(token=-256), dict(head=120), dict(head=8),
         dict(page=1 << 40)]
SHAPES = [
    (dict(dtype=0), INVALID), (dict(dtype=3), INVALID), (dict(B=-1), INVALID), (dict(Hkv=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(page_size=12), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
    (dict(max_pages=1 << 27), UNSUPPORTED), (dict(num_pages=-1), INVALID),
]


def attend(L=None, sh=None, **kw):
    a = dict(shape=shape(**(sh or {})), rule=ctypes.byref(_native.ScoreRule(0.1, 0.0, 0, None)), q=FAKE, qr=4096,
             qp=1024, qh=128, k=pool(), v=pool(0x40000), ks=FAKE, vs=FAKE, block=16, table=FAKE, lens=FAKE,
             nd=None, out=FAKE, lse=None, ws=0x100000, wsb=1 << 30, st=None)
    a.update(kw)
    return sv.library().paged_attention_q8(*a.values())


@pytest.mark.parametrize("sh,status", SHAPES + [
    (dict(P=0), INVALID), (dict(P=18), UNSUPPORTED), (dict(Hq=9), INVALID), (dict(Hq=130), UNSUPPORTED),
    (dict(Hq=66, D=256), UNSUPPORTED), (dict(B=0), OK)])
def test_attention_shapes(sh, status):
    assert attend(sh=sh) == status
    assert (sv.library().paged_attention_q8_workspace(shape(**sh)) > 0) == (status == OK)


@pytest.mark.parametrize("kw,status", [
    *[(dict(k=pool(**p)), INVALID) for p in POOLS], *[(dict(v=pool(**p)), INVALID) for p in POOLS],
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(qr=0), INVALID), (dict(qp=-8), INVALID),
    (dict(qh=4), INVALID), (dict(ks=None), INVALID), (dict(vs=ODD), INVALID), (dict(block=0), INVALID),
    (dict(block=3), INVALID), (dict(block=32), INVALID), (dict(table=None), INVALID),
    (dict(lens=ODD), INVALID), (dict(nd=ODD), INVALID), (dict(out=None), INVALID), (dict(lse=ODD), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=0x100080), WORKSPACE), (dict(wsb=1000), WORKSPACE),
    (dict(rule=None), INVALID), (dict(rule=ctypes.byref(_native.ScoreRule(float("nan"), 0, 0, None))), INVALID),
])
def test_attention_arguments(kw, status):
    assert attend(**kw) == status


def test_blocks_end_at_a_tile():
    assert attend(sh=dict(page_size=1024), block=256) == UNSUPPORTED
    assert append(sh=dict(page_size=1024), block=256) == UNSUPPORTED


def test_the_limit_of_the_waits_is_checked():
    L = sv.library()
    for us in (0, 100001):
        assert L.paged_attention_q8_wait_selftest(*[None] * 3, 0, 0, 0, *[None] * 4, 16, *[None] * 6, 0,
                                                  us, None) == INVALID


def append(sh=None, **kw):
    a = dict(shape=shape(**(sh or {})), rows=5, k=FAKE, kr=256, kh=128, v=FAKE, vr=256, vh=128, slots=FAKE,
             kp=pool(), vp=pool(0x40000), ks=FAKE, vs=FAKE, block=16, st=None)
    a.update(kw)
    return sv.library().kv_cache_append_q8(*a.values())


@pytest.mark.parametrize("sh,status", SHAPES)
def test_append_shapes(sh, status):
    assert append(sh) == status


@pytest.mark.parametrize("kw,status", [
    *[(dict(kp=pool(**p)), INVALID) for p in POOLS], *[(dict(vp=pool(**p)), INVALID) for p in POOLS],
    (dict(rows=-1), INVALID), (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(rows=0, k=None), OK),
    (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(kr=-8), INVALID), (dict(kr=100), INVALID),
    (dict(vh=4), INVALID), (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID),
    (dict(ks=None), INVALID), (dict(vs=ODD), INVALID), (dict(block=0), INVALID), (dict(block=12), INVALID),
    (dict(block=32), INVALID),
])
def test_append_arguments(kw, status):
    assert append(**kw) == status


def page_map(**kw):
    """Every array in a place of its own."""
    a = dict(B=4, page=16, pages=100, table=0x10000, cols=10, olds=0x20000, lens=0x21000, add=0x22000,
             ring=0x30000, size=100, state=0x40000, P=3, rows=12, slots=0x50000, pos=0x51000, out=0x52000,
             first=0x53000, next=0x54000, st=None)
    a.update(kw)
    return sv.library().kv_page_map(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(B=0, P=0, rows=0), OK), (dict(B=8193, P=0), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED), (dict(page=4), UNSUPPORTED), (dict(page=0), INVALID),
    (dict(cols=1 << 26), UNSUPPORTED), (dict(cols=0), INVALID), (dict(pages=-1), INVALID),
    (dict(size=0), INVALID), (dict(P=-1), INVALID), (dict(rows=11), INVALID), (dict(P=0, rows=-1), INVALID),
    *[({x: None}, INVALID) for x in ("table", "olds", "lens", "add", "ring", "state", "slots", "pos", "out",
                                     "first", "next")],
    *[({x: ODD}, INVALID) for x in ("table", "olds", "lens", "add", "ring", "state", "slots", "pos", "out",
                                    "first", "next")],
    (dict(slots=0x50004), INVALID),
    # what other CTAs still read
    (dict(out=0x20000), INVALID), (dict(out=0x21000), INVALID), (dict(out=0x22000), INVALID),
    (dict(out=0x20000 - 12), INVALID), (dict(out=0x2000c), INVALID), (dict(first=0x21004), INVALID),
    (dict(next=0x40000), INVALID), (dict(next=0x40004), INVALID), (dict(next=0x20008), INVALID),
    (dict(out=0x40000), INVALID), (dict(first=0x40000), INVALID),
])
def test_page_map_refusals(kw, status):
    assert page_map(**kw) == status


@pytest.mark.parametrize("kw", [
    # table: 160 bytes, ring: 400, slots: 96, positions: 48, lengths: 16
    dict(table=0x30000 - 156), dict(ring=0x10000 + 156), dict(table=0x20000), dict(ring=0x21000 - 396),
    dict(slots=0x10000 - 88), dict(slots=0x30000 + 392), dict(slots=0x21008), dict(pos=0x22000 + 12),
    dict(pos=0x10000 - 44), dict(pos=0x50000 + 92), dict(pos=0x40004), dict(out=0x50000 + 92),
    dict(out=0x51000 - 12), dict(first=0x52000 - 16), dict(next=0x53000 + 16), dict(next=0x54000, first=0x54000 - 16),
    dict(next=0x30000 + 396), dict(P=0, rows=3, pos=0x50000 + 20),
])
def test_page_map_arrays_that_share_bytes_are_refused(kw):
    assert page_map(**kw) == INVALID


def head_rows(data=FAKE, heads=4, req=1024, row=512, head=128, out=0x90000, oq=1024, orow=512, oh=128, w=None):
    return ctypes.byref(_native.HeadRows(data, req, row, head, out, oq, orow, oh, heads, w))


def rotate(**kw):
    a = dict(dtype=1, B=3, P=2, D=128, R=128, q=head_rows(), k=head_rows(heads=1), w32=1, pos=FAKE, freq=FAKE,
             f64=0, norm=1, eps=1e-6, inter=0, st=None)
    a.update(kw)
    return sv.library().qk_norm_rotate(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), INVALID), (dict(B=-1), INVALID), (dict(P=-1), INVALID), (dict(B=0, pos=None), OK),
    (dict(P=0), OK), (dict(D=96, R=96), UNSUPPORTED), (dict(R=24), UNSUPPORTED), (dict(R=144), UNSUPPORTED),
    (dict(R=-16), INVALID), (dict(B=1 << 16, P=1 << 16), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(pos=None), INVALID), (dict(pos=ODD), INVALID), (dict(freq=None), INVALID), (dict(freq=ODD), INVALID),
    (dict(f64=1, freq=FAKE + 4), INVALID),
    *[(dict(q=head_rows(**x)), INVALID) for x in (
        dict(data=None), dict(data=FAKE + 8), dict(out=None), dict(out=FAKE + 2), dict(heads=-1), dict(req=-8),
        dict(row=4), dict(head=12), dict(oq=0), dict(orow=0), dict(oh=0), dict(w=ODD), dict(oh=1 << 39))],
])
def test_rotate_refusals(kw, status):
    assert rotate(**kw) == status


# ------------------------------------------------------------------------------ the binding
STREAM = SimpleNamespace(cuda_stream=0)


@pytest.fixture
def new():
    if torch.cuda.is_available():
        pytest.skip("fakes stand in for the tensors of a GPU")
    with FakeTensorMode(allow_non_fake_inputs=True):
        yield lambda *s, dtype=torch.bfloat16, device="cuda": torch.empty(s, dtype=dtype, device=device)


def arguments(new):
    i32 = lambda *s: new(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: new(*s, dtype=torch.float32)  # noqa: E731
    i64 = lambda *s: new(*s, dtype=torch.int64)  # noqa: E731
    codes, scales = new(4, 16, 2, 64, dtype=torch.float8_e4m3fn), f32(4, 2, 2)
    return {
        "kv_page_map": dict(page_table=i32(3, 4), old_len=i32(3), seq_len=i32(3), num_new=i32(3), ring=i32(12),
                            ring_state=i32(2), page_size=16, num_pages=12, out_slots=i64(3, 2),
                            out_positions=i32(3, 2), out_len=i32(3), out_first=i32(4), out_state=i32(2)),
        "qk_norm_rotate": dict(q=new(3, 4, 64), k=new(3, 2, 64), positions=i32(3), inv_freq=f32(32),
                               q_weight=f32(64), k_weight=f32(64), out_q=new(3, 4, 64), out_k=new(3, 2, 64)),
        "kv_cache_append_q8": dict(k=new(3, 2, 64), v=new(3, 2, 64), slots=i64(3), k_cache=codes, v_cache=codes,
                                   k_scale=scales, v_scale=scales),
        "paged_attention_q8": dict(q=new(3, 1, 4, 64), k_cache=codes, v_cache=codes, k_scale=scales,
                                   v_scale=scales, page_table=i32(3, 2), seq_len=i32(3), out=new(3, 1, 4, 64),
                                   out_lse=f32(3, 1, 4)),
    }


NAMES = ["kv_page_map", "qk_norm_rotate", "kv_cache_append_q8", "paged_attention_q8"]


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_checked(new, name):
    """Each argument in turn with another type, another size, off the device, or not contiguous where it
    has to be: an error before anything is launched."""
    good = arguments(new)[name]
    call = lambda a: getattr(sv, name)(**a, stream=STREAM)  # noqa: E731
    for key, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = [new(*t.shape, dtype=torch.float64 if t.dtype != torch.float64 else torch.float32),
                 new(*t.shape, dtype=t.dtype, device="cpu"),
                 new(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype),
                 new(*t.shape, 2, dtype=t.dtype)[..., 0], None if key not in ("inv_freq", "q_weight", "k_weight")
                 and not key.startswith("out_") else "text"]
        if key == "ring":  # of any size
            del wrong[2]
        if key == "page_table":  # of any width
            wrong[2] = new(t.shape[0] + 1, t.shape[1], dtype=t.dtype)
        if key == "inv_freq":
            wrong[0], wrong[2] = new(32, dtype=torch.float16), new(33, dtype=torch.float32)
        if name == "qk_norm_rotate" and key in ("q_weight", "k_weight"):
            wrong[0] = new(64, dtype=torch.float16)
        for w in wrong:
            with pytest.raises((TypeError, ValueError, AttributeError, RuntimeError)):
                call({**good, key: w})


@pytest.mark.parametrize("name", NAMES)
def test_a_transformed_tensor_is_refused(new, name):
    """A tensor inside torch.func.vmap has no address: an error, not the end of the process."""
    good = arguments(new)[name]
    key = next(iter(good))
    t = good[key]
    with pytest.raises((RuntimeError, TypeError, ValueError)):
        torch.func.vmap(lambda x: getattr(sv, name)(**{**good, key: x}, stream=STREAM))(
            new(2, *t.shape, dtype=t.dtype))


def test_rows_that_are_not_one_stride_apart_are_refused(new):
    good = arguments(new)["kv_cache_append_q8"]
    slots = new(3, 2, dtype=torch.int64)
    k, apart = new(3, 2, 2, 64), new(3, 3, 2, 64)[:, :2]
    for a in ((k, apart), (apart, k)):
        with pytest.raises(ValueError, match="stride"):
            sv.kv_cache_append_q8(*a, slots, *list(good.values())[3:], stream=STREAM)


def test_rows_or_positions_are_given(new):
    good = arguments(new)["kv_page_map"]
    del good["out_slots"]
    for kw in ({}, dict(P=2, rows=6)):
        with pytest.raises(ValueError, match="rows"):
            sv.kv_page_map(**good, **kw, stream=STREAM)


def test_a_workspace_off_the_device_is_refused(new):
    good = arguments(new)["paged_attention_q8"]
    for ws in (new(1 << 24, dtype=torch.uint8, device="cpu"), new(1 << 21, 8, dtype=torch.uint8)[:, 0], "text"):
        with pytest.raises((TypeError, ValueError)):
            sv.paged_attention_q8(**good, workspace=ws, stream=STREAM)
