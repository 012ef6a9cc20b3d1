"""Attention over 4-bit rows with the largest steps and least values that the format allows
(no data quantises to all of them at once: the rows are made here)."""
import math

import numpy as np
import pytest
import torch

from gpu_util import check_no_device_error
from prefix_ref import check, make as make_prefix, reference as prefix_reference
from q4_ref import D, GROUP, ROW, make, reference
from window_ref import check_out

pytestmark = pytest.mark.gpu

STEP, LEAST = 60.0, 448.0
VMAX = LEAST + 15 * STEP


def extreme_rows(shape, seed):
    """[..., 80] uint8: any codes, s in {0, 60}, m in {-448, 0, 448}."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (*shape, D // 2), dtype=np.uint8)
    s = rng.choice([0.0, STEP, STEP], (*shape, D // GROUP))
    m = rng.choice([-LEAST, 0.0, LEAST], (*shape, D // GROUP))
    parts = np.stack([s, m], -1).astype(np.float16).reshape(*shape, 2 * D // GROUP)
    rows = np.concatenate([codes, np.ascontiguousarray(parts).view(np.uint8)], -1)
    assert rows.shape[-1] == ROW
    return torch.from_numpy(rows).cuda()


def put(c, seed):
    for i, x in enumerate(("key_pages", "value_pages")):
        c[x] = extreme_rows(c[x].shape[:-1], seed + i)
    # scores of a few units, so that the softmax is not one key's
    c["query"] = (c["query"].float() * 2.0 ** -5).to(torch.bfloat16)
    return c


@pytest.mark.parametrize("L,H_q,H_kv", [(1, 8, 2), (1, 28, 4), (5, 8, 2), (40, 8, 2), (300, 8, 2)])
def test_attention(L, H_q, H_kv):
    import paged_kv_attention_06_gb300 as pa
    lens = [L, L + 100, 700]
    c = put(make(lens, H_q, H_kv, L, 16, seed=L, poison=False), seed=L)
    out = pa.pa_attention_q4(**c, max_context_len=max(lens))
    check_no_device_error()
    # Both routes hold the weights P = 2^(s - m) in f16 (the prefill's values are f16 in the
    # reference as well): off by 2^-11 of the weight, or by 2^-25 where that is less than
    # f16's least normal number. The key that set the maximum in use adds 1 to the sum l, so
    # l >= 1 and that is at most 2^-25 |v| of the quotient for each key, whatever the others'
    # values are (they may all be 0 here, which leaves nothing of sum p |v|).
    check_out(out, reference(c, copied=L > 8), True, max(lens), VMAX)
    assert math.isfinite(float(out.float().abs().max()))


def test_behind_a_prefix():
    import paged_kv_attention_06_gb300 as pa
    lens = [400, 401, 600, 450]
    c = put(make_prefix([(400, 4)], lens, 8, 2, 1, D, 16, 3, "q4", poison=False), seed=3)
    out = pa.pa_decode_prefix_q4(**c)
    check_no_device_error()
    check(out, prefix_reference(c, "q4"), "q4", max(lens), VMAX)


def test_what_the_append_writes_is_within_the_bounds():
    import paged_kv_attention_06_gb300 as pa
    x = torch.randn(1, 4, 64, D, device="cuda") * torch.logspace(-8, 38, 64, device="cuda")[:, None]
    x[0, 0, :, ::2] = -3e38
    x[0, 1, :, 1::3] = float("inf")
    kp, vp = (torch.zeros((4, 4, 16, ROW), dtype=torch.uint8, device="cuda") for _ in "kv")
    slots = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    pa.pa_append_kv_q4(x.to(torch.bfloat16), (-x).to(torch.bfloat16), kp, vp, slots, 16)
    check_no_device_error()
    for pool in (kp, vp):
        parts = pool[..., 64:].contiguous().view(torch.float16).float()
        s, m = parts[..., 0::2], parts[..., 1::2]
        assert (s >= 0).all() and (s <= STEP).all() and (m.abs() <= LEAST).all()
        assert float(s.max()) > 59
