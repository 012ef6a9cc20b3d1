"""pa_decode_weights against a plain 64-bit reference: the output as for
pa_decode, and every slot's accumulated weight.

Tolerance of a weight: each row's share p has the relative error of its score
(D truncated fp32 additions: 2^-16 scale sum |q| |k|, once in the numerator and
once in the sum), of the sum of n terms (n 2^-24), of the exponentials and the
product (2^-20); shares are positive, so their sum has no more. The old weight
times decay is rounded twice (2^-23). Shares below fp32's normal range vanish
(1e-37 each).
"""
import pytest
import torch

from gpu_util import check_no_device_error
from window_ref import SCALES, check_out, make, reference

pytestmark = pytest.mark.gpu


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def run(c, wp, decay, fp8=False, causal=True, **kw):
    pa = _pa()
    f = pa.pa_decode_weights_fp8 if fp8 else pa.pa_decode_weights
    extra = dict(k_scale=SCALES[0], v_scale=SCALES[1]) if fp8 else {}
    if "max_context_len" not in kw:
        kw["max_context_len"] = max(1, int(c["context_lens"].max()))
    return f(**c, **extra, weight_pages=wp, decay=decay, causal=causal, **kw)


def pool_like(c, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(c["key_pages"].shape[:3], generator=g, device="cuda")


def check_weights(wp, old, c, ref, decay, L):
    ps = c["page_size"]
    mine = torch.zeros((wp.shape[0], ps), dtype=torch.bool, device="cuda")
    for b, (_, _, size, w) in enumerate(ref):
        n = w.shape[1]
        j = torch.arange(n, device="cuda")
        page, off = c["block_table"][b, j // ps].long(), j % ps
        mine[page, off] = True
        kept = torch.where(j < n - L, old[page, :, off].double().T * decay, 0.0) if decay else torch.zeros_like(w)
        got = wp[page, :, off].double().T
        tol = w * (size * 2.0 ** -15 + n * 2.0 ** -24 + 2.0 ** -20) + kept * 2.0 ** -23 + 1e-34
        err = (got - (kept + w)).abs()
        assert torch.all(err <= tol), (b, float((err / tol).max()))
    # slots behind every context are as they were
    assert torch.equal(wp.transpose(1, 2)[~mine], old.transpose(1, 2)[~mine])


def check(lens, H_q, H_kv, L, D, ps, decay, seed, fp8=False, causal=True):
    c = make(lens, H_q, H_kv, L, D, ps, seed, fp8=fp8)
    wp = pool_like(c, seed)
    old = wp.clone()
    out = run(c, wp, decay, fp8, causal)
    check_no_device_error()
    ref = reference(c, fp8=fp8, causal=causal)
    check_out(out, ref, fp8, max(lens))
    check_weights(wp, old, c, ref, decay, L)


LENS = [0, 1, 2, 17, 63, 64, 65, 130, 500, 1030]


@pytest.mark.parametrize("ps", [1, 4, 16, 64, 256])
@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("decay", [0.0, 0.9, 1.0])
def test_one_row(ps, D, fp8, decay):
    check(LENS, 8, 2, 1, D, ps, decay, seed=ps + D, fp8=fp8)


@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (128, True)])
@pytest.mark.parametrize("L,H_q,H_kv", [(2, 4, 2), (5, 7, 1), (16, 2, 1), (32, 8, 2), (3, 16, 1), (70, 4, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_rows(L, H_q, H_kv, D, fp8, causal):
    check(LENS, H_q, H_kv, L, D, 16, 0.5, seed=L, fp8=fp8, causal=causal)


@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (28, 4), (32, 8), (33, 1)])
def test_head_layouts(H_q, H_kv):
    check([5, 700, 90, 4100], H_q, H_kv, 1, 128, 16, 1.0, seed=H_q)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_contexts(fp8):
    check([40000, 20011], 8, 2, 1, 128, 16, 0.25, seed=3, fp8=fp8)


def test_output_is_pa_decodes():
    """The few-row kernel's output is that of pa_decode_window with a window
    past every context, the many-row kernel's that of pa_decode."""
    pa = _pa()
    c = make([300, 4000, 1], 28, 4, 1, 128, 16, seed=4)
    got = run(c, pool_like(c), 1.0)
    check_out(got, reference(c), False, 4000)
    assert torch.equal(got, pa.pa_decode_window(**c, window=4000, max_context_len=4000))
    c = make([300, 4000, 1], 28, 4, 3, 128, 16, seed=4)
    got = run(c, pool_like(c), 1.0)
    assert torch.equal(got, pa.pa_decode(**c, max_context_len=4000))


def test_decay_zero_reads_no_old_weight():
    c = make(LENS, 4, 2, 3, 64, 16, seed=5)
    wp = torch.full(c["key_pages"].shape[:3], float("nan"), device="cuda")
    run(c, wp, 0.0)
    check_no_device_error()
    zero = torch.zeros_like(wp)
    live = ~torch.isnan(wp)
    zero[live] = wp[live]
    full = torch.where(live, zero, torch.zeros_like(wp))
    check_weights(full, torch.zeros_like(wp), c, reference(c), 0.0, 3)


def test_weights_of_a_row_sum_to_one():
    c = make([777], 4, 2, 5, 128, 16, seed=6)
    wp = torch.zeros(c["key_pages"].shape[:3], device="cuda")
    run(c, wp, 0.0)
    # 2 heads a group, 5 rows: each KV head's slots hold 10 in all
    assert torch.allclose(wp.double().sum((0, 2)), torch.full((2,), 10.0, dtype=torch.float64, device="cuda"),
                          rtol=2.0 ** -12, atol=0)


def test_repeated_calls_give_the_same_bits():
    c = make([3000, 1500, 40], 28, 4, 1, 128, 16, seed=7)
    first = pool_like(c)
    second = first.clone()
    a, b = run(c, first, 0.75), run(c, second, 0.75)
    assert torch.equal(a, b) and torch.equal(first, second)


def test_context_past_the_bound_is_cut_and_recorded():
    pa = _pa()
    c = make([300, 100], 4, 2, 1, 64, 16, seed=8, poison=False)
    wp = pool_like(c)
    old = wp.clone()
    run(c, wp, 1.0, max_context_len=200)
    st, flags = pa.pa_get_device_error()
    assert st == pa.PA_ERR_DEVICE_BOUNDS and flags == pa.PA_DEVERR_CONTEXT_LEN
    page = c["block_table"][0, 13:19].long()                 # positions 208 and on
    assert torch.equal(wp[page], old[page])


def test_refusals():
    pa = _pa()
    c = make([30, 20], 4, 2, 1, 128, 16, seed=9)
    wp = pool_like(c)
    for kw, err in ((dict(decay=-1.0), pa.PagedAttentionError), (dict(decay=float("nan")), pa.PagedAttentionError),
                    (dict(decay=float("inf")), pa.PagedAttentionError),
                    (dict(max_context_len=0), pa.PagedAttentionError),
                    (dict(weight_pages=wp.double()), TypeError), (dict(weight_pages=wp[:, :1]), ValueError),
                    (dict(weight_pages=wp.cpu()), ValueError), (dict(page_size=8), ValueError),
                    (dict(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda")), pa.PagedAttentionError)):
        old = wp.clone()
        with pytest.raises(err):
            pa.pa_decode_weights(**{**dict(c, weight_pages=wp, max_context_len=30), **kw})
        assert torch.equal(wp, old)


def test_other_stream_and_replayed_graph():
    c = make([900, 300, 77], 8, 2, 1, 128, 16, seed=10)
    want = pool_like(c)
    for _ in range(3):
        out = run(c, want, 0.5)
    wp = pool_like(c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = run(c, wp, 0.5, stream=side)
    side.synchronize()
    assert torch.equal(wp, want) and torch.equal(got, out)
    wp.copy_(pool_like(c))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, wp, 0.5, out=got, max_context_len=900)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(wp, want)
