"""Calls from a host thread that has made no CUDA call before: the same results."""
import threading

import pytest
import torch

from window_ref import SCALES, make

pytestmark = pytest.mark.gpu


def case(name):
    """A call that allocates nothing and asks nothing of the device but the call itself."""
    import paged_kv_attention_06_gb300 as pa
    L = 40 if "prefill" in name else 1
    fp8 = name.endswith("e4m3")
    c = make([100, 57], 4, 2, L, 128, 16, seed=3, poison=False, fp8=fp8)
    scales = dict(k_scale=SCALES[0], v_scale=SCALES[1]) if fp8 else {}
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(c["query"])
    more = dict(out=out, workspace=ws, max_context_len=100)
    wp = torch.ones(c["key_pages"].shape[:3], device="cuda")
    if name.startswith("decode"):
        f = pa.pa_decode_fp8 if fp8 else pa.pa_decode
        return out, lambda: f(**c, **scales, **more)
    if name.startswith("window_decode"):
        f = pa.pa_decode_window_fp8 if fp8 else pa.pa_decode_window
        return out, lambda: f(**c, **scales, **more, window=50)
    if name.startswith("weights"):
        f = pa.pa_decode_weights_fp8 if fp8 else pa.pa_decode_weights
        return out, lambda: f(**c, **scales, **more, weight_pages=wp, decay=0.0)
    if name == "prefill":
        return out, lambda: pa.pa_prefill(**c, out=out)
    if name == "split_prefill":
        return out, lambda: pa.pa_prefill_split(**c, out=out, workspace=ws)
    if name == "window_prefill":
        return out, lambda: pa.pa_prefill_window(**c, out=out, window=50)
    if name == "window_prefill_e4m3":
        return out, lambda: pa.pa_attention_window_fp8(**c, **scales, **more, window=50)
    kept = torch.zeros((2, 2, 30), dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert name == "evict"
    return kept, lambda: pa.pa_kv_evict(c["key_pages"], c["value_pages"], wp, c["block_table"], c["context_lens"], 16,
                                        keep=30, kept=kept, new_lens=lens)


@pytest.mark.parametrize("name", ["decode", "decode_e4m3", "window_decode", "window_decode_e4m3", "weights",
                                  "weights_e4m3", "prefill", "split_prefill", "window_prefill", "window_prefill_e4m3",
                                  "evict"])
def test_first_cuda_call_of_a_thread(name):
    out, call = case(name)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    out, call = case(name)                            # other addresses: no tensor map made before fits
    errors = []

    def body():
        try:
            call()
        except Exception as e:
            errors.append(e)

    thread = threading.Thread(target=body)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert torch.equal(out, want)
