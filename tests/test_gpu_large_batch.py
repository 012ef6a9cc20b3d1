"""Window and weight decodes of batches so large that the few-row kernel's table of
requests does not fit beside its rings (pa_decode takes them too), and pa_prefill_window
where the tensor-core kernel cannot run: the split-KV kernel with one tile of query rows.

Against a plain 64-bit reference. Tolerance of an output: bf16 rounding (2^-8 of the
value), the weights rounded for P . V (bf16, 2^-8 of sum p |v|; e4m3 pools f16, twice
2^-11, and 2^-25 of |v| a key where f16 is subnormal), D truncated fp32 additions of a
score (2^-16 of scale sum |q| |k|, on both sides of the quotient). Of a weight: the same
scores, 2^-20 for the exponentials and the products, 2^-23 for old * decay.
"""
import math

import pytest
import torch

from gpu_util import check_no_device_error
from window_ref import F8, SCALES

pytestmark = pytest.mark.gpu


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def batch(B, H_q, H_kv, L, D, fp8, seed, n_max=40, ps=16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-n_max // ps)
    lens = torch.randint(0, n_max + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[:3] = torch.tensor([0, 1, n_max])
    bt = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    kp, vp = (torch.randn((B * width, H_kv, ps, D), generator=g, device="cuda") for _ in "kv")
    if fp8:
        kp, vp = ((x / s).clamp(-448, 448).to(F8).view(torch.uint8) for x, s in zip((kp, vp), SCALES))
    else:
        kp, vp = kp.to(torch.bfloat16), vp.to(torch.bfloat16)
    q = (torch.randn((B, H_q, L, D), generator=g, device="cuda") * 1.3).to(torch.bfloat16)
    return dict(query=q, key_pages=kp, value_pages=vp, block_table=bt, context_lens=lens, page_size=ps)


def check(c, out, fp8, W=None, S=0, weights=None):
    """weights: (pool after, pool before, decay)."""
    B, H_q, L, D = c["query"].shape
    H_kv, ps = c["key_pages"].shape[1:3]
    n = c["context_lens"].long()[:, None]
    j = torch.arange(c["block_table"].shape[1] * ps, device="cuda")
    at = n - L + torch.arange(L, device="cuda")
    see = (j <= at[:, :, None]) & (j < n[:, :, None])
    if W is not None:
        see = see & ((j > at[:, :, None] - W) | (j < S))
    page = c["block_table"][:, j // ps].long()
    assert torch.isfinite(out.float()).all()
    step = max(1, (1 << 27) // (H_kv * len(j) * D * 8))
    for b in range(0, B, step):
        part = slice(b, b + step)
        k, v = (x[page[part], :, j % ps].transpose(1, 2) for x in (c["key_pages"], c["value_pages"]))
        if fp8:
            k, v = k.view(F8).float().double() * SCALES[0], v.view(F8).float().double() * SCALES[1]
        k, v = k.double(), v.double()                           # [b, H_kv, n, D]
        q = c["query"][part].double().view(len(k), H_kv, -1, D)  # rows (head, i)
        seen = see[part][:, None].repeat(1, H_q // H_kv, 1, 1).view(len(k), 1, -1, len(j))
        z = (q @ k.transpose(2, 3) / math.sqrt(D)).masked_fill(~seen, -math.inf)
        p = torch.softmax(z, -1).nan_to_num(0.0)
        size = float((q.abs() @ k.abs().transpose(2, 3)).max()) / math.sqrt(D)
        r, mag = (p @ v).view(out[part].shape), (p @ v.abs()).view(out[part].shape)
        tol = r.abs() * 2.0 ** -8 + mag * ((2.0 ** -10 if fp8 else 2.0 ** -8) + size * 2.0 ** -15) + 1e-30
        if fp8:
            tol = tol + len(j) * 2.0 ** -25 * 448 * SCALES[1]
        assert torch.all((out[part].double() - r).abs() <= tol)
        if weights is not None:
            pool, old, decay = weights
            w = p.sum(2)                                        # [b, H_kv, n]
            got, was = (x[page[part], :, j % ps].transpose(1, 2).double() for x in (pool, old))
            new = torch.where((j < n[part] - L)[:, None], was * decay, 0.0)
            tol = w * (size * 2.0 ** -15 + 2.0 ** -20) + new * 2.0 ** -23 + 1e-34
            live = (j < n[part])[:, None]
            assert torch.all(((got - (new + w)).abs() <= tol) | ~live)
            assert torch.all((got == was) | live)               # slots behind stay


# (head_dim, rows a KV group, requests): past the few-row kernel's table, within pa_decode's
SIZES = [(128, 1, 14000), (128, 16, 12500), (64, 4, 20000)]


@pytest.mark.parametrize("D,R,B", SIZES)
def test_window_decode(D, R, B):
    pa = _pa()
    c = batch(B, R, 1, 1, D, False, seed=B)
    full = pa.pa_decode(**c, max_context_len=40)
    check_no_device_error()
    check(c, full, False)
    out = pa.pa_decode_window(**c, window=9, sinks=2, max_context_len=40)
    check_no_device_error()
    check(c, out, False, 9, 2)


@pytest.mark.parametrize("D,R,B", SIZES)
def test_weights(D, R, B):
    pa = _pa()
    c = batch(B, R, 1, 1, D, False, seed=B + 1)
    pool = torch.rand(c["key_pages"].shape[:3], device="cuda")
    old = pool.clone()
    out = pa.pa_decode_weights(**c, weight_pages=pool, max_context_len=40, decay=0.5)
    check_no_device_error()
    check(c, out, False, weights=(pool, old, 0.5))


def test_e4m3_pools():
    pa = _pa()
    c = batch(14000, 2, 1, 1, 128, True, seed=5)
    ks, vs = SCALES
    out = pa.pa_decode_window_fp8(**c, k_scale=ks, v_scale=vs, window=9, sinks=2, max_context_len=40)
    check_no_device_error()
    check(c, out, True, 9, 2)
    pool = torch.rand(c["key_pages"].shape[:3], device="cuda")
    old = pool.clone()
    out = pa.pa_decode_weights_fp8(**c, weight_pages=pool, k_scale=ks, v_scale=vs, max_context_len=40)
    check_no_device_error()
    check(c, out, True, weights=(pool, old, 1.0))


def test_a_batch_past_both_tables_is_unsupported():
    pa = _pa()
    c = batch(30000, 1, 1, 1, 128, False, seed=6)
    pool = torch.rand(c["key_pages"].shape[:3], device="cuda")
    for f in (lambda: pa.pa_decode(**c), lambda: pa.pa_decode_window(**c, window=9),
              lambda: pa.pa_decode_weights(**c, weight_pages=pool, max_context_len=40)):
        with pytest.raises(pa.PagedAttentionError) as e:
            f()
        assert e.value.status == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H_q,H_kv,L", [(1, 1, 1), (8, 2, 4), (2, 2, 5), (8, 2, 8), (4, 1, 40)])
@pytest.mark.parametrize("W,S", [(5, 0), (17, 3)])
def test_window_prefill_without_the_tensor_core_kernel(D, H_q, H_kv, L, W, S):
    pa = _pa()
    c = batch(7, H_q, H_kv, L, D, False, seed=L, n_max=150)
    pa.pa_debug_prefill_variant(7)
    try:
        out = pa.pa_prefill_window(**c, window=W, sinks=S)
    finally:
        pa.pa_debug_prefill_variant(0)
    check_no_device_error()
    check(c, out, False, W, S)


def test_the_largest_e4m3_batches_run_or_are_unsupported():
    """The table of requests, up to the last that fits beside the e4m3 kernel's own arrays."""
    pa = _pa()
    c = batch(32000, 1, 1, 1, 128, True, seed=7, n_max=16)
    ws = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["query"])

    def runs(B):
        part = {k: x[:B] if k in ("query", "block_table", "context_lens") else x for k, x in c.items()}
        try:
            pa.pa_decode_fp8(**part, k_scale=1.0, v_scale=1.0, out=out[:B], max_context_len=16, workspace=ws)
        except pa.PagedAttentionError as e:
            assert e.status == pa.PA_ERR_UNSUPPORTED, (B, e)
            return False
        return True

    lo, hi = 1, 32000                                # runs, does not
    assert runs(lo) and not runs(hi)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if runs(mid) else (lo, mid)
    for B in range(lo - 40, lo + 100):
        assert runs(B) == (B <= lo)
    check_no_device_error()
