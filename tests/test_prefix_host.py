"""Argument checks of the decode behind shared prefixes through the C ABI, without a
GPU: a bad call is refused before anything is looked up or launched."""
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
    tables, tail = [vp] * 5 + [i32, f32], [vp] * 3 + [i32] * 3 + [vp, Shape, i32, vp, sz, vp]
    lib.pa_decode_prefix.argtypes = lib.pa_decode_prefix_q4.argtypes = tables + tail
    lib.pa_decode_prefix_fp8.argtypes = tables + [f32, f32] + tail
    for n in ("", "_fp8", "_q4"):
        f = getattr(lib, f"pa_decode_prefix{n}_workspace_bytes")
        f.argtypes, f.restype = [Shape, i32, i32, i32], sz
    return lib


GOOD = dict(q=0x10000, k=0x20000, v=0x30000, bt=0x40000, cl=0x50000, ps=16, scale=0.1, ks=1.0, vs=1.0,
            pt=0x80000, pl=0x90000, pst=0xA0000, np=1, pp=4, mpl=60, out=0x60000, mcl=100, ws=0x70000, wsb=1 << 30)
SHAPE = dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, q_len=1, num_pages=64, max_pages=8)


def args_of(bad):
    a = dict(GOOD, **{k: v for k, v in bad.items() if k != "shape"})
    return a, Shape(**dict(SHAPE, **bad.get("shape", {})))


def calls(lib, a, s):
    t = [a[k] for k in ("q", "k", "v", "bt", "cl", "ps", "scale")]
    tail = [a[k] for k in ("pt", "pl", "pst", "np", "pp", "mpl", "out")] + [s, a["mcl"], a["ws"], a["wsb"], None]
    yield lib.pa_decode_prefix(*t, *tail)
    yield lib.pa_decode_prefix_q4(*t, *tail)
    yield lib.pa_decode_prefix_fp8(*t, a["ks"], a["vs"], *tail)


@pytest.mark.parametrize("bad,expect", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1), (dict(cl=None), 1),
    (dict(out=None), 1), (dict(pt=None), 1), (dict(pl=None), 1), (dict(pst=None), 1), (dict(q=0x10002), 1),
    (dict(k=0x20008), 1), (dict(out=0x60004), 1), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1),
    (dict(pp=0), 1), (dict(pp=-2), 1), (dict(ps=12), 2), (dict(ps=512), 2), (dict(pp=1 << 28), 2),
    (dict(shape=dict(batch=0)), 1), (dict(shape=dict(q_len=0)), 1), (dict(shape=dict(num_pages=0)), 1),
    (dict(shape=dict(max_pages=0)), 1), (dict(shape=dict(head_dim=96)), 2), (dict(shape=dict(num_q_heads=5)), 2),
    (dict(shape=dict(num_pages=1 << 30)), 2),
])
def test_refusals(lib, bad, expect):
    a, s = args_of(bad)
    assert list(calls(lib, a, s)) == [expect] * 3


@pytest.mark.parametrize("bad", [dict(ks=0.0), dict(vs=-1.0), dict(ks=float("nan")), dict(vs=float("inf"))])
def test_scales(lib, bad):
    a, s = args_of(bad)
    assert list(calls(lib, a, s))[2] == 1


def test_workspace_of_invalid_sizes_is_zero(lib):
    for f in (lib.pa_decode_prefix_workspace_bytes, lib.pa_decode_prefix_fp8_workspace_bytes,
              lib.pa_decode_prefix_q4_workspace_bytes):
        for bad in (dict(head_dim=96), dict(batch=0), dict(num_q_heads=5), dict(q_len=0)):
            assert f(Shape(**dict(SHAPE, **bad)), 16, 1, 60) == 0
        for ps, count, longest in ((12, 1, 60), (16, 0, 60), (16, 257, 60), (16, 1, 0), (16, 1, 1 << 30)):
            assert f(Shape(**SHAPE), ps, count, longest) == 0
