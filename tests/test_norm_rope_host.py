"""Argument checks of pa_qk_norm_rope_append through the C ABI, without a GPU:
a bad call is refused before anything is looked up or launched."""
import ctypes

import pytest


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "num_q_heads", "num_kv_heads", "head_dim", "q_len", "num_pages",
                 "max_pages")]


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_06_gb300 import build
    lib = ctypes.CDLL(build.build())
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    qk = [vp, i64, i64, vp, vp, f32, vp, i32, i32, ctypes.c_int, vp, vp, vp, vp, vp, i32]
    lib.pa_qk_norm_rope_append.argtypes = qk + [Shape, vp]
    lib.pa_qk_norm_rope_append_fp8.argtypes = qk + [f32, f32, Shape, vp]
    return lib


GOOD = dict(qkv=0x10000, bs=8 * 128 * 3, ts=8 * 128, qw=0x20000, kw=0x21000, eps=1e-6, cs=0x30000,
            R=128, T=16, inter=0, pos=0x40000, q=0x50000, kp=0x60000, vp=0x70000, sm=0x80000,
            ps=16)
SHAPE = dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, q_len=3, num_pages=4,
             max_pages=0)


@pytest.mark.parametrize("bad,expect", [
    (dict(qkv=None), 1), (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1),
    (dict(sm=None), 1), (dict(qkv=0x10008), 1), (dict(q=0x50002), 1), (dict(kp=0x60004), 1),
    (dict(qw=0x20008), 1), (dict(cs=0x30004), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(cs=None), 1), (dict(pos=None), 1), (dict(T=0), 1), (dict(R=-16), 1), (dict(R=144), 1),
    (dict(R=24), 2), (dict(ps=12), 2), (dict(ps=512), 2),
    (dict(ts=8 * 128 + 4), 1), (dict(ts=7 * 128), 1), (dict(bs=-8), 1), (dict(bs=8), 1),
    (dict(shape=dict(batch=0)), 1), (dict(shape=dict(q_len=-1)), 1),
    (dict(shape=dict(num_pages=0)), 1), (dict(shape=dict(head_dim=192), bs=8 * 192 * 3, ts=8 * 192), 2),
    (dict(shape=dict(num_q_heads=5)), 2),
])
def test_refusals(lib, bad, expect):
    a = dict(GOOD, **{k: v for k, v in bad.items() if k != "shape"})
    s = Shape(**dict(SHAPE, **bad.get("shape", {})))
    args = [a[k] for k in ("qkv", "bs", "ts", "qw", "kw", "eps", "cs", "R", "T", "inter", "pos",
                           "q", "kp", "vp", "sm", "ps")]
    assert lib.pa_qk_norm_rope_append(*args, s, None) == expect
    assert lib.pa_qk_norm_rope_append_fp8(*args, 1.0, 1.0, s, None) == expect


@pytest.mark.parametrize("scales", [(0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0),
                                    (1.0, float("inf"))])
def test_bad_scales(lib, scales):
    args = [GOOD[k] for k in ("qkv", "bs", "ts", "qw", "kw", "eps", "cs", "R", "T", "inter", "pos",
                              "q", "kp", "vp", "sm", "ps")]
    assert lib.pa_qk_norm_rope_append_fp8(*args, *scales, Shape(**SHAPE), None) == 1


def test_e4m3_head_dim_64_is_unsupported(lib):
    args = [GOOD[k] for k in ("qkv", "bs", "ts", "qw", "kw", "eps", "cs", "R", "T", "inter", "pos",
                              "q", "kp", "vp", "sm", "ps")]
    args[7] = 64
    s = Shape(**dict(SHAPE, head_dim=64))
    assert lib.pa_qk_norm_rope_append_fp8(*args, 1.0, 1.0, s, None) == 2
