"""Rows whose query is NaN come out as NaN from every attention call, however their keys are
split between blocks and warps, and keys that are NaN make NaN of the rows that see them; all
other rows stay finite."""
import pytest
import torch

from gpu_util import check_no_device_error
from q4_ref import make
from window_ref import F8, SCALES

pytestmark = pytest.mark.gpu


def batch(lens, L, kind, H_q=8, H_kv=2):
    c = make(lens, H_q, H_kv, L, 16, seed=L, poison=False)
    g = torch.Generator(device="cuda").manual_seed(L)
    if kind != "q4":
        for x, s in zip(("key_pages", "value_pages"), SCALES):
            t = torch.randn((*c[x].shape[:-1], 128), generator=g, device="cuda")
            c[x] = t.to(torch.bfloat16) if kind == "bf16" else (t / s).clamp(-448, 448).to(F8).view(torch.uint8)
    return c


def calls(kind, most):
    import paged_kv_attention_06_gb300 as pa
    s = dict(k_scale=SCALES[0], v_scale=SCALES[1])
    return {
        "bf16": [lambda c: pa.pa_decode(**c), lambda c: pa.pa_prefill(**c),
                 lambda c: pa.pa_attention(**c, max_context_len=most),
                 lambda c: pa.pa_attention_window(**c, window=100, sinks=4)],
        "e4m3": [lambda c: pa.pa_decode_fp8(**c, **s), lambda c: pa.pa_prefill_fp8(**c, **s, max_context_len=most),
                 lambda c: pa.pa_attention_window_fp8(**c, **s, window=100, sinks=4)],
        "q4": [lambda c: pa.pa_decode_q4(**c), lambda c: pa.pa_prefill_q4(**c, max_context_len=most)],
    }[kind]


def check(out, nan):
    check_no_device_error()
    assert out[nan].isnan().all()
    assert out[~nan].isfinite().all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("L", [1, 5, 16, 40, 300])
@pytest.mark.parametrize("extra", [0, 400, 20000])
def test_queries(L, extra, kind):
    c = batch([L + extra, L + extra + 3], L, kind)
    nan = torch.zeros(2, 8, L, dtype=torch.bool, device="cuda")
    nan[0, 3, L - 1] = nan[1, 6, 0] = True
    c["query"][nan] = float("nan")
    for f in calls(kind, L + extra + 3):
        check(f(c), nan)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("n", [1, 64, 65, 129, 4097])
def test_the_last_key(n, kind):
    """Alone in its tile, or in its warp's, where n is one past a whole number of them."""
    c = batch([n, n], 1, kind)
    page, at = c["block_table"][0, (n - 1) // 16].item(), (n - 1) % 16
    c["key_pages"][page, 0, at] = float("nan") if kind == "bf16" else {"e4m3": 0x7F, "q4": 0xFF}[kind]
    nan = torch.zeros(2, 8, 1, dtype=torch.bool, device="cuda")
    nan[0, :4] = True
    for f in calls(kind, n):
        check(f(c), nan)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("n", [65, 129, 4097])
def test_a_value_that_one_row_sees(n, kind):
    """The last value is NaN, in a tile that the chunk's other rows see nothing of."""
    import paged_kv_attention_06_gb300 as pa
    c = batch([n, n], 2, kind)
    page, at = c["block_table"][0, (n - 1) // 16].item(), (n - 1) % 16
    c["value_pages"][page, 0, at] = float("nan") if kind == "bf16" else {"e4m3": 0x7F, "q4": 0xFF}[kind]
    f = {"bf16": pa.pa_decode, "q4": pa.pa_decode_q4}.get(kind)
    out = f(**c) if f else pa.pa_decode_fp8(**c, k_scale=SCALES[0], v_scale=SCALES[1])
    check_no_device_error()
    assert out[0, :4, 1].isnan().all() and out[0, 4:].isfinite().all() and out[1].isfinite().all()
    if kind == "bf16":                       # one key a block's piece: the first row's piece is empty
        assert out[0, :4, 0].isfinite().all()
