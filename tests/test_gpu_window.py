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
    c = make([1, 64, 777, 2100], 8, 2, 3, 128, 16, seed=3, poison=False)
    got = pa.pa_decode_window(**c, window=W, sinks=7)
    want = pa.pa_decode(**c)
    assert torch.equal(got, want)


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
