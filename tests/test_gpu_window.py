"""Sliding-window decode with sink tokens against a plain 64-bit reference, at
the sizes, masks and page layouts where it can go wrong. Slots that no row
sees hold NaN and pages that no row sees have table entry -1."""
import pytest
import torch

from gpu_util import check_no_device_error
from window_ref import SCALES, check_out, make, reference

pytestmark = pytest.mark.gpu


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def run_decode(c, W, S, fp8=False, **kw):
    pa = _pa()
    f = pa.pa_decode_window_fp8 if fp8 else pa.pa_decode_window
    extra = dict(k_scale=SCALES[0], v_scale=SCALES[1]) if fp8 else {}
    return f(**c, **extra, window=W, sinks=S, **kw)


def check_decode(lens, H_q, H_kv, L, D, ps, W, S, seed, fp8=False, mcl=True):
    c = make(lens, H_q, H_kv, L, D, ps, seed, W, S, fp8)
    out = run_decode(c, W, S, fp8, max_context_len=max(lens) if mcl else 0)
    check_no_device_error()
    check_out(out, reference(c, W, S, fp8), fp8, W + S + L)


LENS = [0, 1, 2, 17, 63, 64, 65, 127, 128, 200, 333, 1000, 1025, 2500]


@pytest.mark.parametrize("ps", [1, 2, 4, 8, 16, 64, 128, 256])
@pytest.mark.parametrize("W,S", [(1, 0), (1, 1), (63, 4), (64, 64), (100, 0), (129, 65), (512, 4)])
def test_one_row(ps, W, S):
    check_decode(LENS, 8, 2, 1, 128, ps, W, S, seed=ps + W)


@pytest.mark.parametrize("ps", [1, 16, 64, 256])
@pytest.mark.parametrize("W,S", [(1, 0), (63, 4), (100, 16), (513, 65)])
@pytest.mark.parametrize("H_q,H_kv", [(7, 1), (4, 4), (16, 1)])
def test_one_row_e4m3(H_q, H_kv, ps, W, S):
    check_decode(LENS, H_q, H_kv, 1, 128, ps, W, S, seed=ps + W + H_q, fp8=True)


@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("L,H_q,H_kv", [(2, 4, 2), (5, 7, 1), (16, 2, 1), (24, 8, 2), (3, 16, 1), (70, 4, 4)])
@pytest.mark.parametrize("W,S", [(1, 3), (40, 4), (300, 0)])
def test_several_rows(L, H_q, H_kv, W, S, D, fp8):
    check_decode(LENS, H_q, H_kv, L, D, 16, W, S, seed=L + W, fp8=fp8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (28, 4), (32, 8), (33, 1)])
def test_head_layouts(H_q, H_kv, D):
    check_decode([5, 700, 90, 4100], H_q, H_kv, 1, D, 16, 256, 4, seed=H_q + D)


@pytest.mark.parametrize("W", [5000, 1 << 30, 2**31 - 1])
def test_window_past_every_context_is_full_attention(W):
    pa = _pa()
    # 12 rows a group: the few-row kernel, which rounds P less than pa_decode's
    c = make([1, 64, 777, 2100], 8, 2, 3, 128, 16, seed=3, poison=False)
    got = pa.pa_decode_window(**c, window=W, sinks=7)
    check_out(got, reference(c), False, 2100)
    # 20 rows: pa_decode's kernel, the same bits
    c = make([1, 64, 777, 2100], 8, 2, 5, 128, 16, seed=3, poison=False)
    assert torch.equal(pa.pa_decode_window(**c, window=W, sinks=7), pa.pa_decode(**c))


@pytest.mark.parametrize("S", [90, 5000, 2**31 - 1])
def test_sinks_that_reach_the_window_or_past_the_context(S):
    check_decode([10, 100, 150, 700], 4, 2, 2, 64, 8, 64, S, seed=4)


def test_unknown_max_context_len_and_many_requests():
    check_decode([(37 * i) % 1500 for i in range(200)], 8, 8, 1, 64, 16, 100, 4, seed=5, mcl=False)


def test_long_context_reads_the_window_alone():
    n = 200000
    check_decode([n, n - 77], 8, 2, 1, 128, 16, 1024, 4, seed=6)
    check_decode([n, n - 77], 8, 2, 1, 128, 64, 1024, 4, seed=6, fp8=True)


def test_offsets_past_32_bits():
    """Rows whose byte offset in the pool is past 2^32."""
    pa = _pa()
    c = make([500], 4, 2, 1, 128, 16, seed=7, W=100, S=4)
    P = (1 << 24) // 32 + 64                     # 2^24 rows of 256 bytes, and 64 pages more
    used = c["key_pages"].shape[0]
    for x in ("key_pages", "value_pages"):
        big = torch.full((P, 2, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        big[P - used:] = c[x]
        c[x] = big
    c["block_table"][c["block_table"] >= 0] += P - used
    out = pa.pa_decode_window(**c, window=100, sinks=4)
    check_no_device_error()
    check_out(out, reference(c, 100, 4), False, 200)


def test_bad_page_and_length_are_recorded():
    pa = _pa()
    c = make([300, 200], 4, 2, 1, 64, 16, seed=8, W=64, S=4, poison=False)
    c["block_table"][0, 300 // 16] = 1 << 20
    pa.pa_decode_window(**c, window=64, sinks=4)
    assert pa.pa_get_device_error() == (pa.PA_ERR_DEVICE_BOUNDS, pa.PA_DEVERR_PAGE_ID)
    c = make([300, 200], 4, 2, 1, 64, 16, seed=8, W=64, S=4, poison=False)
    c["context_lens"][1] = 16 * c["block_table"].shape[1] + 1
    pa.pa_decode_window(**c, window=64, sinks=4)
    st, flags = pa.pa_get_device_error()
    assert st == pa.PA_ERR_DEVICE_BOUNDS and flags & pa.PA_DEVERR_CONTEXT_LEN


def test_refusals():
    pa = _pa()
    c = make([30, 20], 4, 2, 1, 128, 16, seed=9)
    for kw, err in ((dict(window=0), pa.PagedAttentionError), (dict(window=-4), pa.PagedAttentionError),
                    (dict(sinks=-1), pa.PagedAttentionError), (dict(scale=0.0), pa.PagedAttentionError),
                    (dict(page_size=8), ValueError), (dict(query=c["query"].float()), TypeError),
                    (dict(query=c["query"].cpu()), ValueError),
                    (dict(out=c["query"][:1]), ValueError),
                    (dict(block_table=c["block_table"].cpu()), ValueError),
                    (dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24)), ValueError),
                    (dict(workspace=torch.empty(16, dtype=torch.uint8)), ValueError),
                    (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), pa.PagedAttentionError)):
        with pytest.raises(err):
            pa.pa_decode_window(**{**dict(c, window=8), **kw})
    with pytest.raises(TypeError):                 # bf16 pools through the e4m3 form
        pa.pa_decode_window_fp8(**c, k_scale=1.0, v_scale=1.0, window=8)


def test_two_calls_on_two_streams_and_a_replayed_graph():
    pa = _pa()
    cs = [make([900, 300, 77], 8, 2, 1, 128, 16, seed=20 + i, W=128, S=4) for i in range(2)]
    want = [run_decode(c, 128, 4) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = [run_decode(c, 128, 4, stream=s) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    graphs, outs = [], []
    for c in cs:
        outs.append(torch.empty_like(c["query"]))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run_decode(c, 128, 4, out=outs[-1])
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.zero_()
        torch.cuda.synchronize()


# ---- the prefill kernel and the dispatch ------------------------------------

def run_prefill(c, W, S):
    return _pa().pa_prefill_window(**c, window=W, sinks=S)


def check_prefill(lens, H_q, H_kv, L, D, ps, W, S, seed):
    c = make(lens, H_q, H_kv, L, D, ps, seed, W, S)
    out = run_prefill(c, W, S)
    check_no_device_error()
    check_out(out, reference(c, W, S), False, W + S + 1)


PREFILL_LENS = [0, 1, 60, 128, 129, 300, 1000]


@pytest.mark.parametrize("ps", [1, 2, 4, 8, 16, 64, 128, 256])
@pytest.mark.parametrize("W,S", [(1, 0), (1, 2), (64, 4), (128, 128), (129, 0), (200, 130), (513, 17)])
def test_prefill_pages_and_windows(ps, W, S):
    check_prefill(PREFILL_LENS, 4, 2, 60, 128, ps, W, S, seed=ps + W)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [1, 2, 127, 128, 129, 257, 700])
@pytest.mark.parametrize("W,S", [(40, 4), (300, 0)])
def test_prefill_lengths(L, W, S, D):
    check_prefill([0, 3, L, L + 1, L + 200, L + 999], 4, 2, L, D, 16, W, S, seed=L + D)


@pytest.mark.parametrize("ps", [4, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (3, 1), (7, 1), (28, 4), (8, 8), (32, 8)])
def test_prefill_head_layouts(H_q, H_kv, D, ps):
    check_prefill([100, 431], H_q, H_kv, 100, D, ps, 90, 5, seed=H_q + D)


def test_prefill_many_items_per_block_and_many_tiles():
    check_prefill([40 + (13 * i) % 700 for i in range(90)], 8, 2, 40, 64, 16, 64, 4, seed=30)
    check_prefill([6000, 5500], 32, 8, 5000, 128, 16, 257, 4, seed=31)


@pytest.mark.parametrize("W", [100000, 2**31 - 1])
def test_prefill_window_past_every_context_is_full_attention(W):
    pa = _pa()
    c = make([130, 64, 777, 2100], 8, 2, 130, 128, 16, seed=32, poison=False)
    assert torch.equal(run_prefill(c, W, 3), pa.pa_prefill(**c))


@pytest.mark.parametrize("L", [1, 24, 25, 32, 33, 200])
@pytest.mark.parametrize("mcl", [0, 4200])
def test_dispatch(L, mcl):
    pa = _pa()
    c = make([L, L + 300, 4200], 8, 2, L, 128, 16, 33, W=200, S=4)
    got = pa.pa_attention_window(**c, window=200, sinks=4, max_context_len=mcl)
    check_no_device_error()
    check_out(got, reference(c, 200, 4), False, 300)
    if L <= 24:
        assert torch.equal(got, run_decode(c, 200, 4, max_context_len=mcl))
    else:
        # without room for the split kernel: pa_prefill_window
        none = torch.empty(16, dtype=torch.uint8, device="cuda")
        got = pa.pa_attention_window(**c, window=200, sinks=4, max_context_len=mcl, workspace=none)
        assert torch.equal(got, run_prefill(c, 200, 4))


@pytest.mark.parametrize("ps", [1, 16, 128, 256])
@pytest.mark.parametrize("L", [3, 9, 130, 300])
@pytest.mark.parametrize("W,S", [(1, 0), (100, 4), (300, 130), (5000, 4)])
def test_dispatch_e4m3(L, W, S, ps):
    pa = _pa()
    lens = [0, 2, L, L + 77, L + 1500]
    c = make(lens, 7, 1, L, 128, ps, 34, W, S, fp8=True)
    got = pa.pa_attention_window_fp8(**c, k_scale=SCALES[0], v_scale=SCALES[1], window=W, sinks=S,
                                     max_context_len=max(lens))
    check_no_device_error()
    # the second route rounds P to bf16
    ref = reference(c, W, S, fp8=True)
    check_out(got, ref, L <= 8, min(W, 3000) + S + L)


def test_e4m3_copies_hold_the_seen_tokens_alone():
    """The workspace of a short window over a long context is small, and the
    longest context a bound allows works with it."""
    pa = _pa()
    c = make([60000, 59993], 4, 1, 100, 128, 16, 35, W=256, S=4, fp8=True)
    shape = pa.make_shape(c["query"].shape, c["key_pages"].shape, c["block_table"].shape[1])
    need = pa.pa_attention_window_fp8_workspace_bytes(shape, 16, 60000, 256, 4)
    assert need < 2 * 6 * 128 * 128 * 2 * 2 + 2 * 469 * 4
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got = pa.pa_attention_window_fp8(**c, k_scale=SCALES[0], v_scale=SCALES[1], window=256, sinks=4,
                                     max_context_len=60000, workspace=ws)
    check_no_device_error()
    check_out(got, reference(c, 256, 4, fp8=True), False, 400)


def test_prefill_and_dispatch_refusals():
    pa = _pa()
    c = make([300, 200], 4, 2, 100, 128, 16, seed=36)
    for kw, err in ((dict(window=0), pa.PagedAttentionError), (dict(sinks=-1), pa.PagedAttentionError),
                    (dict(scale=float("inf")), pa.PagedAttentionError), (dict(page_size=8), ValueError)):
        with pytest.raises(err):
            pa.pa_prefill_window(**{**dict(c, window=8), **kw})
        with pytest.raises(err):
            pa.pa_attention_window(**{**dict(c, window=8), **kw})
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_attention_window(**c, window=8, max_context_len=-1)
    c = make([300, 200], 4, 2, 100, 128, 16, seed=36, fp8=True)
    ok = dict(c, k_scale=1.0, v_scale=1.0, window=8, max_context_len=300)
    for kw in (dict(k_scale=0.0), dict(v_scale=float("nan")), dict(window=-1), dict(sinks=-1),
               dict(workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(pa.PagedAttentionError):
            pa.pa_attention_window_fp8(**{**ok, **kw})


def test_prefill_bad_page_is_recorded():
    pa = _pa()
    c = make([300, 200], 4, 2, 100, 64, 16, seed=37, W=64, S=4, poison=False)
    c["block_table"][0, 300 // 16] = 1 << 20
    run_prefill(c, 64, 4)
    assert pa.pa_get_device_error() == (pa.PA_ERR_DEVICE_BOUNDS, pa.PA_DEVERR_PAGE_ID)


def test_prefill_replayed_graph_on_another_stream():
    c = make([300, 700], 8, 2, 200, 128, 16, seed=38, W=128, S=4)
    want = run_prefill(c, 128, 4)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _pa().pa_prefill_window(**c, window=128, sinks=4, out=out)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---- the prefill with its tiles spread over the SMs ---------------------------

@pytest.fixture
def split_always():
    """Test setting 6: the split kernel for every windowed prefill that it can
    take, in pieces of about two tiles."""
    pa = _pa()
    pa.pa_debug_prefill_variant(6)
    yield
    pa.pa_debug_prefill_variant(0)


def check_split(lens, H_q, H_kv, L, ps, W, S, seed, fp8=False):
    pa = _pa()
    c = make(lens, H_q, H_kv, L, 128, ps, seed, W, S, fp8)
    mcl = max(max(lens), 1)
    shape = pa.make_shape(c["query"].shape, c["key_pages"].shape, c["block_table"].shape[1])
    ref = reference(c, W, S, fp8)
    if fp8:
        c.update(k_scale=SCALES[0], v_scale=SCALES[1])
        need = pa.pa_attention_window_fp8_workspace_bytes(shape, ps, mcl, W, S)
        call = pa.pa_attention_window_fp8
    else:
        need = pa.pa_attention_window_workspace_bytes(shape, ps, mcl, W, S)
        assert need > 0
        call = pa.pa_attention_window
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = call(**c, window=W, sinks=S, max_context_len=mcl, workspace=ws)
    check_no_device_error()
    check_out(out, ref, False, W + S + 1)
    again = call(**c, window=W, sinks=S, max_context_len=mcl, workspace=ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("ps", [8, 16, 64, 128, 256])
@pytest.mark.parametrize("W,S", [(1, 0), (1, 2), (64, 4), (128, 128), (129, 0), (200, 130), (513, 17), (5000, 4)])
def test_split_pages_and_windows(split_always, ps, W, S):
    check_split(PREFILL_LENS, 4, 2, 60, ps, W, S, seed=ps + W)


@pytest.mark.parametrize("L", [40, 127, 128, 129, 257, 700])
@pytest.mark.parametrize("W,S", [(40, 4), (300, 0), (900, 20)])
def test_split_lengths(split_always, L, W, S):
    check_split([0, 3, L, L + 1, L + 200, L + 999], 4, 2, L, 16, W, S, seed=L + W)


@pytest.mark.parametrize("H_q,H_kv", [(2, 1), (3, 1), (7, 1), (28, 4), (32, 8)])
def test_split_head_layouts(split_always, H_q, H_kv):
    check_split([100, 1431], H_q, H_kv, 100, 16, 490, 5, seed=H_q)


@pytest.mark.parametrize("L", [9, 130])
@pytest.mark.parametrize("W,S", [(100, 4), (300, 130), (1000, 0)])
def test_split_e4m3(split_always, L, W, S):
    check_split([0, 2, L, L + 77, L + 1500], 8, 2, L, 16, W, S, seed=34, fp8=True)


def test_split_of_few_items_and_long_windows():
    """Shapes that the call itself spreads over the SMs: many pieces an item,
    and two items a block short of two rounds."""
    check_split([6000], 8, 2, 100, 16, 4096, 4, seed=50)
    check_split([4500, 5200], 32, 8, 600, 16, 2048, 20, seed=51)


def test_split_in_a_replayed_graph_sees_new_inputs():
    pa = _pa()
    c, fresh = (make([6000], 8, 2, 100, 128, 16, s, 4096, 4, poison=False) for s in (52, 53))
    kw = dict(window=4096, sinks=4, max_context_len=6000)
    shape = pa.make_shape(c["query"].shape, c["key_pages"].shape, c["block_table"].shape[1])
    need = pa.pa_attention_window_workspace_bytes(shape, 16, 6000, 4096, 4)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["query"])
    pa.pa_attention_window(**c, **kw, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_attention_window(**c, **kw, out=out, workspace=ws)
    graph.replay()
    want = pa.pa_attention_window(**fresh, **kw, workspace=torch.zeros_like(ws))
    for k in ("query", "key_pages", "value_pages", "block_table"):
        c[k].copy_(fresh[k])
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
