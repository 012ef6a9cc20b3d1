"""Argument checks of the 4-bit calls through the C ABI, without a GPU: a bad call is
refused before anything is looked up or launched."""
import ctypes

import pytest

vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t


class Shape(ctypes.Structure):
    _fields_ = [(n, i32) for n in
                ("batch", "num_q_heads", "num_kv_heads", "head_dim", "q_len", "num_pages",
                 "max_pages")]


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_06_gb300 import build
    lib = ctypes.CDLL(build.build())
    attn = [vp] * 5 + [i32, f32, ctypes.c_int, vp, Shape, i32, vp, sz, vp]
    lib.pa_decode_q4.argtypes = lib.pa_prefill_q4.argtypes = lib.pa_attention_q4.argtypes = attn
    lib.pa_append_kv_q4.argtypes = [vp] * 5 + [i32, Shape, vp]
    lib.pa_gather_kv_q4.argtypes = [vp] * 4 + [i32, Shape, i32, vp, vp, vp]
    lib.pa_decode_q4_workspace_bytes.argtypes = [Shape]
    lib.pa_decode_q4_workspace_bytes.restype = sz
    for f in (lib.pa_prefill_q4_workspace_bytes, lib.pa_attention_q4_workspace_bytes):
        f.argtypes, f.restype = [Shape, i32], sz
    return lib


GOOD = dict(q=0x10000, k=0x20000, v=0x30000, bt=0x40000, cl=0x50000, ps=16, scale=0.1, causal=1, out=0x60000,
            mcl=100, ws=0x70000, wsb=1 << 30, x=0x80000, y=0x90000, len=100)
SHAPE = dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, q_len=1, num_pages=64, max_pages=8)


def args_of(bad):
    a = dict(GOOD, **{k: v for k, v in bad.items() if k != "shape"})
    return a, Shape(**dict(SHAPE, **bad.get("shape", {})))


@pytest.mark.parametrize("L", [1, 400])
@pytest.mark.parametrize("bad,expect", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1), (dict(cl=None), 1),
    (dict(out=None), 1), (dict(q=0x10002), 1), (dict(k=0x20008), 1), (dict(v=0x30004), 1), (dict(out=0x60004), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(ps=12), 2), (dict(ps=512), 2),
    (dict(shape=dict(batch=0)), 1), (dict(shape=dict(q_len=0)), 1), (dict(shape=dict(num_pages=0)), 1),
    (dict(shape=dict(max_pages=0)), 1), (dict(shape=dict(head_dim=64)), 2), (dict(shape=dict(head_dim=96)), 2),
    (dict(shape=dict(num_q_heads=5)), 2), (dict(shape=dict(num_pages=1 << 30)), 2),
])
def test_attention_refusals(lib, bad, expect, L):
    a, s = args_of(bad)
    if "q_len" not in bad.get("shape", {}):
        s.q_len = L
    for f in (lib.pa_decode_q4, lib.pa_prefill_q4, lib.pa_attention_q4):
        assert f(*[a[k] for k in ("q", "k", "v", "bt", "cl", "ps", "scale", "causal", "out")], s, a["mcl"], a["ws"],
                 a["wsb"], None) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1),
    (dict(x=0x80008), 1), (dict(y=0x90002), 1), (dict(k=0x20008), 1), (dict(v=0x30001), 1),
    (dict(ps=0), 2), (dict(ps=3), 2), (dict(shape=dict(batch=0)), 1), (dict(shape=dict(q_len=-1)), 1),
    (dict(shape=dict(num_pages=0)), 1), (dict(shape=dict(head_dim=64)), 2), (dict(shape=dict(num_pages=1 << 30)), 2),
])
def test_append_refusals(lib, bad, expect):
    a, s = args_of(bad)
    assert lib.pa_append_kv_q4(a["x"], a["y"], a["k"], a["v"], a["bt"], a["ps"], s, None) == expect


@pytest.mark.parametrize("bad,expect", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1),
    (dict(cl=None), 1), (dict(x=0x80008), 1), (dict(k=0x20008), 1), (dict(len=0), 1), (dict(len=-3), 1),
    (dict(ps=0), 2), (dict(ps=3), 2), (dict(shape=dict(batch=0)), 1), (dict(shape=dict(max_pages=0)), 1),
    (dict(shape=dict(head_dim=64)), 2), (dict(shape=dict(num_pages=1 << 30)), 2),
    (dict(len=2**31 - 1, shape=dict(batch=1 << 20)), 2),
])
def test_gather_refusals(lib, bad, expect):
    a, s = args_of(bad)
    assert lib.pa_gather_kv_q4(a["k"], a["v"], a["bt"], a["cl"], a["ps"], s, a["len"], a["x"], a["y"], None) == expect


def test_workspace_of_invalid_shapes_is_zero(lib):
    for bad in (dict(head_dim=64), dict(batch=0), dict(num_q_heads=5), dict(q_len=0)):
        s = Shape(**dict(SHAPE, **bad))
        assert lib.pa_decode_q4_workspace_bytes(s) == 0
        assert lib.pa_attention_q4_workspace_bytes(s, 100) == 0
