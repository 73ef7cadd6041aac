"""Planned steps, the rotary write by slots and sparse attention: what the C calls refuse, without a GPU.

The calls check their arguments before any CUDA call, so they are given a pool description of zeros with the sizes
filled in, on a device that does not exist: a call that passes its checks stops there."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def k():
    import paged_kv_cache_kvc_gb300 as k
    if not os.path.exists(k.LIB_PATH):
        from paged_kv_cache_kvc_gb300 import build
        build.build()
    k.load()
    return k


class Fields(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("bs", ctypes.c_int32), ("L", ctypes.c_int32), ("H_KV", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("s", ctypes.c_int32), ("device", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("rest", ctypes.c_uint8 * 4096)]


def pool(bs=16, D=128, H_KV=2):
    return Fields(N=10, bs=bs, L=2, H_KV=H_KV, D=D, dtype=0, s=2, device=-7, bits=16)


P = 4096   # an aligned address that nothing reads


def call(k, name, order, good, change):
    args = {**good, **change}
    at = args.pop("pool", None) or pool()
    return getattr(k.load(), name)(ctypes.byref(at) if at != "none" else None, *[args[x] for x in order.split()])


def check(k, name, order, good, cases):
    stopped = (k.KVC_ERR_ARG, k.KVC_ERR_CUDA)   # at the device: a wrong one, or none at all
    assert call(k, name, order, good, {}) in stopped
    for change, want in cases:
        got = call(k, name, order, good, change)
        assert got == want, (name, change, k.kvc_status_str(got))


def test_plan_step(k):
    order = "bt mb lens new B free cap count lens_out count_out cu slots pos seq rows stream"
    good = dict(bt=P, mb=4, lens=P, new=P, B=3, free=P, cap=10, count=P, lens_out=P, count_out=P, cu=P, slots=P, pos=P, seq=P,
                rows=8, stream=None)
    A, U = k.KVC_ERR_ARG, k.KVC_ERR_UNSUPPORTED
    cases = [({x: None}, A) for x in "bt lens new free count lens_out count_out cu slots".split()]
    cases += [({x: P + 2}, A) for x in "bt lens new free count lens_out count_out cu slots pos seq".split()]
    cases += [(dict(B=-1), A), (dict(B=32769), U), (dict(mb=0), A), (dict(mb=-1), A), (dict(cap=9), A), (dict(cap=2 ** 31), A),
              (dict(rows=-1), A), (dict(rows=2 ** 31), A), (dict(pool="none"), A)]
    check(k, "kvc_plan_step", order, good, cases)


def test_rope_write_slots(k):
    rope = k.kvc_rope(128, 0, P, None, None, 1e-6, 0)
    order = "layer slots pos stride axes axis_of rows q qs H k ks v vs rope out stream"
    far = 1 << 30
    good = dict(layer=0, slots=P, pos=P, stride=4, axes=3, axis_of=P, rows=4, q=far, qs=1024, H=4, k=2 * far, ks=1024, v=3 * far,
                vs=1024, rope=ctypes.byref(rope), out=5 * far, stream=None)
    A, U = k.KVC_ERR_ARG, k.KVC_ERR_UNSUPPORTED
    cases = [({x: None}, A) for x in "slots pos q k v rope out".split()] + [({x: P + 2}, A) for x in "slots pos q k v out".split()]
    cases += [(dict(layer=2), A), (dict(layer=-1), A), (dict(axes=0), A), (dict(axes=9), A), (dict(stride=-1), A), (dict(rows=-1), A),
              (dict(qs=504), A), (dict(ks=255), A), (dict(vs=260), A), (dict(H=-1), A), (dict(out=2 * far), A), (dict(out=far), A),
              (dict(out=3 * far + 64), A), (dict(rope=ctypes.byref(k.kvc_rope(24, 0, P, None, None, 1e-6, 0))), U),
              (dict(rope=ctypes.byref(k.kvc_rope(144, 0, P, None, None, 1e-6, 0))), A),
              (dict(rope=ctypes.byref(k.kvc_rope(64, 0, None, None, None, 1e-6, 0))), A), (dict(rows=0), k.KVC_OK),
              (dict(pool="none"), A)]
    check(k, "kvc_rope_write_slots", order, good, cases)


def test_bounds(k):
    n = ctypes.c_uint64()
    assert k.load().kvc_bounds_bytes(ctypes.byref(pool()), ctypes.byref(n)) == k.KVC_OK
    assert n.value == 2 * (-(-10 * 2 * 260 // 256) * 256)
    assert k.load().kvc_bounds_bytes(None, ctypes.byref(n)) == k.KVC_ERR_ARG
    assert k.load().kvc_bounds_bytes(ctypes.byref(pool()), None) == k.KVC_ERR_ARG
    A = k.KVC_ERR_ARG
    good = dict(layer=0, slots=P, rows=4, bounds=P, bytes=n.value, stream=None)
    check(k, "kvc_update_bounds", "layer slots rows bounds bytes stream", good,
          [(dict(slots=None), A), (dict(slots=P + 1), A), (dict(bounds=None), A), (dict(bounds=P + 128), A),
           (dict(bytes=n.value - 1), A), (dict(layer=2), A), (dict(layer=-1), A), (dict(rows=-1), A), (dict(rows=0), k.KVC_OK),
           (dict(pool="none"), A)])


def test_select_blocks(k):
    A, U = k.KVC_ERR_ARG, k.KVC_ERR_UNSUPPORTED
    order = "layer bounds bytes q H bt mb B seq pos rows top sink recent out stream"
    good = dict(layer=0, bounds=P, bytes=1 << 20, q=P, H=8, bt=P, mb=4, B=3, seq=P, pos=P, rows=5, top=4, sink=1, recent=1, out=P,
                stream=None)
    cases = [({x: None}, A) for x in "bounds q bt pos out".split()] + [({x: P + 2}, A) for x in "bounds q bt pos seq out".split()]
    cases += [(dict(H=7), A), (dict(H=0), A), (dict(H=66), U), (dict(layer=2), A), (dict(bytes=100), A), (dict(mb=0), A),
              (dict(mb=262145), U), (dict(B=-1), A), (dict(seq=None), A), (dict(top=0), A), (dict(top=1), A), (dict(top=65537), A),
              (dict(sink=-1), A), (dict(recent=0), A), (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), A), (dict(rows=-1), A),
              (dict(rows=0), k.KVC_OK), (dict(pool="none"), A)]
    check(k, "kvc_select_blocks", order, good, cases)


def test_sparse_attn(k):
    A, U = k.KVC_ERR_ARG, k.KVC_ERR_UNSUPPORTED
    order = "layer q H bt mb B seq pos rows lists top out lse scale stream"
    good = dict(layer=0, q=P, H=8, bt=P, mb=4, B=3, seq=P, pos=P, rows=5, lists=P, top=4, out=P, lse=P, scale=1.0, stream=None)
    cases = [({x: None}, A) for x in "q bt pos lists out".split()]
    cases += [({x: P + 2}, A) for x in "q bt pos seq lists out lse".split()]
    cases += [(dict(H=7), A), (dict(H=0), A), (dict(H=66), U), (dict(layer=2), A), (dict(mb=0), A), (dict(B=-1), A), (dict(seq=None), A),
              (dict(top=0), A), (dict(top=65537), A), (dict(out=P + 16), A), (dict(scale=0.0), A), (dict(scale=-1.0), A),
              (dict(scale=float("nan")), A), (dict(scale=float("inf")), A), (dict(rows=-1), A), (dict(rows=2 ** 28), A),
              (dict(rows=0), k.KVC_OK), (dict(pool=pool(bs=24)), U), (dict(pool="none"), A)]
    check(k, "kvc_sparse_attn", order, good, cases)


def test_a_rope_with_axes_shows_them_and_keeps_them(k):
    import torch
    axes = torch.zeros(8, dtype=torch.uint8)
    rope = k.Rope(torch.ones(8), axis_of=axes)
    assert rope.axis_of is axes and k.Rope(torch.ones(8)).axis_of is None
    with pytest.raises(AttributeError):
        rope.axis_of = None
