"""Argument checks of the sliding-window and weight-accumulating calls through
the C ABI, without a GPU: a bad call is refused before anything is looked up or
launched."""
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
    tables, tail = [vp] * 5 + [i32, f32], [vp, Shape, i32, vp, sz, vp]
    lib.pa_decode_window.argtypes = lib.pa_attention_window.argtypes = tables + [i32, i32] + tail
    lib.pa_decode_window_fp8.argtypes = tables + [f32, f32, i32, i32] + tail
    lib.pa_attention_window_fp8.argtypes = lib.pa_decode_window_fp8.argtypes
    lib.pa_prefill_window.argtypes = tables + [i32, i32, vp, Shape, vp]
    wtables = [vp] * 6 + [i32, f32]
    lib.pa_decode_weights.argtypes = wtables + [ctypes.c_int, f32] + tail
    lib.pa_decode_weights_fp8.argtypes = wtables + [f32, f32, ctypes.c_int, f32] + tail
    for n in ("window", "window_fp8"):
        f = getattr(lib, f"pa_attention_{n}_workspace_bytes")
        f.argtypes, f.restype = [Shape, i32, i32, i32, i32], sz
    lib.pa_decode_weights_workspace_bytes.argtypes = [Shape, i32]
    lib.pa_decode_weights_workspace_bytes.restype = sz
    lib.pa_decode_window_workspace_bytes.argtypes = [Shape]
    lib.pa_decode_window_workspace_bytes.restype = sz
    return lib


GOOD = dict(q=0x10000, k=0x20000, v=0x30000, w=0x80000, bt=0x40000, cl=0x50000, ps=16, scale=0.1,
            ks=1.0, vs=1.0, W=64, S=4, causal=1, decay=1.0, out=0x60000, mcl=100, ws=0x70000, wsb=1 << 30)
SHAPE = dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, q_len=1, num_pages=64, max_pages=8)

COMMON = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1), (dict(cl=None), 1),
    (dict(out=None), 1), (dict(q=0x10002), 1), (dict(k=0x20008), 1), (dict(out=0x60004), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(ps=12), 2), (dict(ps=512), 2),
    (dict(shape=dict(batch=0)), 1), (dict(shape=dict(q_len=0)), 1), (dict(shape=dict(num_pages=0)), 1),
    (dict(shape=dict(max_pages=0)), 1), (dict(shape=dict(head_dim=96)), 2),
    (dict(shape=dict(num_q_heads=5)), 2), (dict(shape=dict(num_pages=1 << 30)), 2),
]
SCALES = [dict(ks=0.0), dict(vs=-1.0), dict(ks=float("nan")), dict(vs=float("inf"))]


def args_of(bad):
    a = dict(GOOD, **{k: v for k, v in bad.items() if k != "shape"})
    return a, Shape(**dict(SHAPE, **bad.get("shape", {})))


def window_calls(lib, a, s):
    t = [a[k] for k in ("q", "k", "v", "bt", "cl", "ps", "scale")]
    win, tail = [a["W"], a["S"]], [a["out"], s, a["mcl"], a["ws"], a["wsb"], None]
    yield lib.pa_decode_window(*t, *win, *tail)
    yield lib.pa_attention_window(*t, *win, *tail)
    yield lib.pa_prefill_window(*t, *win, a["out"], s, None)
    yield lib.pa_decode_window_fp8(*t, a["ks"], a["vs"], *win, *tail)
    yield lib.pa_attention_window_fp8(*t, a["ks"], a["vs"], *win, *tail)


@pytest.mark.parametrize("L", [1, 400])
@pytest.mark.parametrize("bad,expect", COMMON + [(dict(W=0), 1), (dict(W=-5), 1), (dict(S=-1), 1)])
def test_window_refusals(lib, bad, expect, L):
    a, s = args_of(bad)
    if "q_len" not in bad.get("shape", {}):
        s.q_len = L
    # a route that cannot be chosen is an invalid argument too
    want = {1} if s.q_len == 0 else {expect}
    for st in window_calls(lib, a, s):
        assert st in want


def weight_calls(lib, a, s):
    t = [a[k] for k in ("q", "k", "v", "w", "bt", "cl", "ps", "scale")]
    tail = [a["out"], s, a["mcl"], a["ws"], a["wsb"], None]
    yield lib.pa_decode_weights(*t, a["causal"], a["decay"], *tail)
    yield lib.pa_decode_weights_fp8(*t, a["ks"], a["vs"], a["causal"], a["decay"], *tail)


@pytest.mark.parametrize("bad,expect", COMMON + [
    (dict(w=None), 1), (dict(w=0x80002), 1), (dict(decay=-0.5), 1), (dict(decay=float("nan")), 1),
    (dict(decay=float("inf")), 1), (dict(mcl=0), 1), (dict(mcl=-3), 1)])
def test_weight_refusals(lib, bad, expect):
    a, s = args_of(bad)
    for st in weight_calls(lib, a, s):
        assert st == expect


@pytest.mark.parametrize("bad", SCALES)
def test_bad_scales(lib, bad):
    a, s = args_of(bad)
    for L in (1, 400):
        s.q_len = L
        assert list(window_calls(lib, a, s))[3:] == [1, 1]
    s.q_len = 1
    assert list(weight_calls(lib, a, s))[1] == 1


def test_e4m3_head_dim_64_is_unsupported(lib):
    a, s = args_of(dict(shape=dict(head_dim=64)))
    for L in (1, 400):
        s.q_len = L
        assert list(window_calls(lib, a, s))[3:] == [2, 2]
    s.q_len = 1
    assert list(weight_calls(lib, a, s))[1] == 2


def test_workspace_sizes_of_invalid_calls_are_zero(lib):
    good = Shape(**SHAPE)
    for f in (lib.pa_attention_window_workspace_bytes, lib.pa_attention_window_fp8_workspace_bytes):
        for bad in ((12, 100, 64, 4), (16, -1, 64, 4), (16, 100, 0, 4), (16, 100, 64, -1)):
            assert f(good, *bad) == 0
        assert f(Shape(**dict(SHAPE, q_len=0)), 16, 100, 64, 4) == 0
    assert lib.pa_decode_weights_workspace_bytes(good, 0) == 0
    assert lib.pa_decode_weights_workspace_bytes(Shape(**dict(SHAPE, head_dim=96)), 100) == 0
    assert lib.pa_decode_window_workspace_bytes(Shape(**dict(SHAPE, num_q_heads=3))) == 0
