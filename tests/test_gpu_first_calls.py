"""First calls of a kernel from two host threads at once, with batches of different size:
the kernel's shared-memory limit depends on neither's."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# In a process of its own: each kernel has only one first call.
SCRIPT = r"""
import threading
import torch
import paged_kv_attention_06_gb300 as pa

def call_of(B, H_q, L, D, fp8, mode):
    kp, vp = (torch.zeros((B, 1, 16, D), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in "kv")
    c = dict(query=torch.zeros((B, H_q, L, D), dtype=torch.bfloat16, device="cuda"), key_pages=kp, value_pages=vp,
             block_table=torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(),
             context_lens=torch.full((B,), 3, dtype=torch.int32, device="cuda"), page_size=16)
    if fp8:
        c.update(k_scale=1.0, v_scale=1.0)
    shape = pa.make_shape(c["query"].shape, kp.shape, 1)
    if mode == "full":
        ws = torch.empty(pa.pa_decode_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
        f = pa.pa_decode_fp8 if fp8 else pa.pa_decode
        return lambda s: f(**c, out=torch.empty_like(c["query"]), max_context_len=16, workspace=ws, stream=s)
    if mode == "window":
        ws = torch.empty(pa.pa_decode_window_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
        f = pa.pa_decode_window_fp8 if fp8 else pa.pa_decode_window
        return lambda s: f(**c, window=2, max_context_len=16, workspace=ws, stream=s)
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(shape, 16), dtype=torch.uint8, device="cuda")
    wp = torch.zeros((B, 1, 16), device="cuda")
    f = pa.pa_decode_weights_fp8 if fp8 else pa.pa_decode_weights
    return lambda s: f(**c, weight_pages=wp, max_context_len=16, workspace=ws, stream=s)

streams = [torch.cuda.Stream() for _ in range(2)]
bad = []
for mode in ("full", "window", "weights"):
    for D, fp8 in ((64, False), (128, False), (128, True)):
        for rows in (4, 12, 24, 60):
            pair = [call_of(B, rows, 1, D, fp8, mode) for B in (1, 2500)]
            torch.cuda.synchronize()
            gate = threading.Barrier(2)
            def go(f, s):
                torch.cuda.set_device(0)
                gate.wait()
                try:
                    f(s)
                except pa.PagedAttentionError as e:
                    bad.append((mode, D, fp8, rows, str(e)))
            threads = [threading.Thread(target=go, args=x) for x in zip(pair, streams)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
            torch.cuda.synchronize()
            for f, s in zip(pair, streams):
                try:
                    f(s)
                except pa.PagedAttentionError as e:
                    bad.append(("again", mode, D, fp8, rows, str(e)))
            torch.cuda.synchronize()
assert not bad, bad
print("ok")
"""


def test_first_calls_of_two_batch_sizes_at_once():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(2):
        r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
