"""pa_kv_evict's argument checks through the C ABI, pa_kv_cache_truncate and
pa_kv_cache_trim_window, without a GPU."""
import ctypes

import numpy as np
import pytest


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("batch", "num_q_heads", "num_kv_heads", "head_dim", "q_len", "num_pages",
                 "max_pages")]


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_06_gb300 import build
    lib = ctypes.CDLL(build.build())
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    ev = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, Shape, vp]
    lib.pa_kv_evict.argtypes = ev
    lib.pa_kv_evict_fp8.argtypes = ev
    return lib


GOOD = dict(kp=0x10000, vp=0x20000, wp=0x30000, bt=0x40000, cl=0x50000, ps=16, keep=40, sinks=4,
            recent=8, dst=0x60000, dmp=3, kept=0x70000, nl=0x80000)
SHAPE = dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, q_len=1, num_pages=64,
             max_pages=8)


@pytest.mark.parametrize("bad,expect", [
    (dict(kp=None), 1), (dict(vp=None), 1), (dict(wp=None), 1), (dict(bt=None), 1),
    (dict(cl=None), 1), (dict(dst=None), 1), (dict(kept=None), 1), (dict(nl=None), 1),
    (dict(kp=0x10008), 1), (dict(vp=0x20004), 1), (dict(wp=0x30002), 1),
    (dict(keep=0), 1), (dict(keep=-1), 1), (dict(sinks=-1), 1), (dict(recent=-2), 1),
    (dict(sinks=33), 1), (dict(recent=37), 1), (dict(sinks=2**31 - 1, recent=2**31 - 1), 1),
    (dict(dmp=2), 1), (dict(dmp=0), 1), (dict(ps=24), 2), (dict(ps=512), 2),
    (dict(nl=0x50000), 1), (dict(nl=0x40000), 1), (dict(kept=0x50000 - 300), 1),
    (dict(kept=0x60008), 1), (dict(kept=0x80000 - 4), 1),
    (dict(shape=dict(batch=0)), 1), (dict(shape=dict(num_kv_heads=0)), 1),
    (dict(shape=dict(max_pages=0)), 1), (dict(shape=dict(head_dim=96)), 2),
    (dict(shape=dict(num_pages=1 << 30)), 2),
])
def test_refusals(lib, bad, expect):
    a = dict(GOOD, **{k: v for k, v in bad.items() if k != "shape"})
    s = Shape(**dict(SHAPE, **bad.get("shape", {})))
    args = [a[k] for k in ("kp", "vp", "wp", "bt", "cl", "ps", "keep", "sinks", "recent", "dst",
                           "dmp", "kept", "nl")]
    assert lib.pa_kv_evict(*args, s, None) == expect
    assert lib.pa_kv_evict_fp8(*args, s, None) == expect


def test_e4m3_head_dim_64_is_unsupported(lib):
    args = [GOOD[k] for k in ("kp", "vp", "wp", "bt", "cl", "ps", "keep", "sinks", "recent", "dst",
                              "dmp", "kept", "nl")]
    assert lib.pa_kv_evict_fp8(*args, Shape(**dict(SHAPE, head_dim=64)), None) == 2


@pytest.mark.parametrize("ps", [1, 4, 16])
def test_truncate_gives_back_the_pages_behind(ps):
    import paged_kv_attention_06_gb300 as pa
    c = pa.KVCache(40, ps)
    c.add(7)
    c.add(8)
    n = 8 * ps + (1 if ps > 1 else 0)
    bt, _, _ = c.plan([7, 8], [n, 2], 20, n)
    free = c.free_pages
    row = [p for p in bt[0] if p >= 0]
    for cut in (n, 5 * ps, 4 * ps + (1 if ps > 1 else 0), 0):
        c.truncate(7, cut)
        held = -(-cut // ps)
        assert c.context_len(7) == cut
        assert c.free_pages == free + len(row) - held
    assert c.context_len(8) == 2
    c.truncate(7, 0)
    # the pages come back, and the next tokens start a new page of position 0
    bt, cl, sm = c.plan([7], [3], 20, 3)
    assert list(cl) == [3] and sm[0, 0] % ps == 0
    c.release(7)
    c.release(8)
    assert c.free_pages == 40


def test_truncate_then_append_continues_in_the_tail_page():
    import paged_kv_attention_06_gb300 as pa
    c = pa.KVCache(8, 4)
    c.add(1)
    bt, _, _ = c.plan([1], [14], 8, 14)
    c.truncate(1, 6)
    bt2, cl, sm = c.plan([1], [1], 8, 1)
    assert list(bt2[0, :2]) == list(bt[0, :2]) and list(bt2[0, 2:]) == [-1] * 6
    assert cl[0] == 7 and sm[0, 0] == bt[0, 1] * 4 + 2


def test_truncate_refusals_and_snapshot():
    import paged_kv_attention_06_gb300 as pa
    c = pa.KVCache(8, 4)
    c.add(1)
    c.plan([1], [10], 8, 10)
    for seq, n in ((2, 0), (1, 11), (1, -1)):
        with pytest.raises(pa.PagedAttentionError) as e:
            c.truncate(seq, n)
        assert e.value.status == pa.PA_ERR_INVALID_ARG
        assert c.context_len(1) == 10 and c.free_pages == 5
    snap = c.snapshot()
    c.truncate(1, 3)
    assert c.free_pages == 7
    c.restore(snap)
    assert c.context_len(1) == 10 and c.free_pages == 5
    bt, cl, sm = c.plan([1], [1], 8, 1)
    assert cl[0] == 11 and np.all(bt[0, :3] >= 0)


@pytest.mark.parametrize("ps", [1, 4, 16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (20, 3), (20, 16), (33, 1), (1000, 4)])
def test_trim_window_keeps_what_later_rows_see(ps, window, sinks):
    import paged_kv_attention_06_gb300 as pa
    c = pa.KVCache(200, ps)
    c.add(1)
    rows = {}
    n = 0
    for step in (1, 7, 30, 1, 1, 45, 1):
        bt, cl, sm = c.plan([1], [step], 120, 45)
        n += step
        assert cl[0] == n
        # every key that the step's rows see is in a page the request holds, in
        # the slot it was written to
        for t in range(n - step, n):
            rows[t] = sm[0, t - (n - step)]
        for p in range(n - step, n):
            for j in range(n):
                if j <= p and (j > p - window or j < sinks):
                    assert bt[0, j // ps] * ps + j % ps == rows[j]
        c.trim_window(1, window, sinks)
        held = 200 - c.free_pages
        seen = [j for j in range(n) if j > n - window or j < sinks]
        need = {j // ps for j in seen} | ({n // ps} if n % ps else set())
        assert held == len(need)
        c.trim_window(1, window, sinks)              # again: nothing more
        assert held == 200 - c.free_pages
    snap = c.snapshot()
    c.release(1)
    assert c.free_pages == 200
    c.restore(snap)
    assert c.free_pages == 200 - held and c.context_len(1) == n


def test_trim_window_refusals_and_truncate_after_it():
    import paged_kv_attention_06_gb300 as pa
    c = pa.KVCache(16, 4)
    c.add(1)
    c.plan([1], [30], 16, 30)
    for args in ((2, 4, 0), (1, 0, 0), (1, -1, 0), (1, 4, -1)):
        with pytest.raises(pa.PagedAttentionError) as e:
            c.trim_window(*args)
        assert e.value.status == pa.PA_ERR_INVALID_ARG
    assert c.free_pages == 8
    c.trim_window(1, 6, 4)                           # pages 1 .. 5 (positions 4 .. 23) go
    assert c.free_pages == 13
    with pytest.raises(pa.PagedAttentionError):      # would go on inside a freed page
        c.truncate(1, 10)
    assert c.context_len(1) == 30 and c.free_pages == 13
    c.truncate(1, 8)                                 # at a page border
    assert c.free_pages == 15
    bt, cl, sm = c.plan([1], [1], 16, 1)
    assert cl[0] == 9 and list(bt[0, :3] >= 0) == [True, False, True]
