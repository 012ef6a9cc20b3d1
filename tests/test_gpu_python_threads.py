"""The compiled calls (_pagedattn_calls) and other Python threads: a launch that waits for
room in its stream's queue must not hold the interpreter lock meanwhile."""
import ctypes
import threading
import time

import pytest
import torch

from window_ref import make

pytestmark = pytest.mark.gpu


def sleep_on(stream, seconds):
    """Holds up the stream on the host for a while, in C (usleep), without the
    interpreter lock."""
    from paged_kv_attention_06_gb300 import build
    lib = ctypes.CDLL(build.LIB)                 # with the CUDA runtime that it links
    lib.cudaLaunchHostFunc.argtypes = [ctypes.c_void_p] * 3
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p)
    assert lib.cudaLaunchHostFunc(stream.cuda_stream, usleep, int(seconds * 1e6)) == 0


def calls():
    import paged_kv_attention_06_gb300 as pa
    c = make([100, 37], 4, 2, 1, 128, 16, seed=1, poison=False)
    out, ws = torch.empty_like(c["query"]), torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    wp = torch.ones(c["key_pages"].shape[:3], device="cuda")
    qkv = torch.randn(2, 1, 8 * 128, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    kept = torch.empty(2, 2, 64, dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    return {
        "append": lambda: pa.pa_qk_norm_rope_append(qkv, None, None, None, None, c["key_pages"], c["value_pages"],
                                                    slots, 16, query=out),
        "window": lambda: pa.pa_decode_window(**c, window=50, out=out, workspace=ws, max_context_len=100),
        "weights": lambda: pa.pa_decode_weights(**c, weight_pages=wp, max_context_len=100, out=out, workspace=ws),
        "evict": lambda: pa.pa_kv_evict(c["key_pages"], c["value_pages"], wp, c["block_table"], c["context_lens"], 16,
                                        keep=64, kept=kept, new_lens=lens),
    }


@pytest.mark.parametrize("kind", ["append", "window", "weights", "evict"])
def test_a_launch_that_waits_lets_other_threads_run(kind):
    call = calls()[kind]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    thread = threading.Thread(target=tick)
    thread.start()
    sleep_on(stream, 0.8)
    start = time.perf_counter()
    with torch.cuda.stream(stream):
        for _ in range(4000):
            call()
    end = time.perf_counter()
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    if end - start < 0.7:
        pytest.skip("the queue took all launches: none had to wait")
    assert max(b - a for a, b in zip(ticks, ticks[1:])) < 0.3
