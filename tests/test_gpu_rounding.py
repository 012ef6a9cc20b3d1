"""How far the window and weight decodes round, at inputs that show it.

Few rows over bf16 pages: the weights p go into P . V as two bf16 parts, whose sum is
within 2^-16 of p. One part alone (2^-8 of each p) is hidden where the output is as large
as its own rounding, so here the values are chosen orthogonal to the weights: the output
is next to nothing and every rounding of P stands alone. Each query has one element that
is not 0, so a score is one exact product.

e4m3 pages: p is one f16, 2^-11 of p, or 2^-25 of the largest weight in use where p is
subnormal; that largest is no larger than the true one, so over the sum l of the weights
relative to the true largest the second part is at most 2^-25 sum |v| / l. More than 16 rows: a warp's O / l
in f16 too, 2^-11 of it or 2^-25 v_scale.

Sums: a lane adds at most every 32nd weight to l (2^-24 each); a warp's products come in
steps of 16 keys, of which it has at most every fourth (2^-22 each, truncated).
"""
import math

import pytest
import torch

from gpu_util import check_no_device_error
from window_ref import F8, SCALES, make

pytestmark = pytest.mark.gpu


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def decode(c, kind, fp8, **kw):
    pa = _pa()
    scales = dict(k_scale=SCALES[0], v_scale=SCALES[1]) if fp8 else {}
    n = int(c["context_lens"].max())
    if kind == "window":
        f = pa.pa_decode_window_fp8 if fp8 else pa.pa_decode_window
        return f(**c, **scales, window=n, sinks=3, max_context_len=n, **kw)
    f = pa.pa_decode_weights_fp8 if fp8 else pa.pa_decode_weights
    wp = torch.zeros(c["key_pages"].shape[:3], device="cuda")
    return f(**c, **scales, weight_pages=wp, decay=0.0, max_context_len=n, **kw)


@pytest.mark.parametrize("kind", ["window", "weights"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R", [1, 4, 7, 8, 12, 16])
@pytest.mark.parametrize("n", [64, 150, 700])
def test_few_rows_keep_sixteen_bits_of_a_weight(kind, D, R, n):
    ps, pages = 16, -(-n // 16)
    g = torch.Generator(device="cuda").manual_seed(n + R + D)
    bt = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    j = torch.arange(n, device="cuda")
    page = bt[0, j // ps].long()
    q = torch.zeros((1, R, 1, D), dtype=torch.bfloat16, device="cuda")
    r = torch.arange(R, device="cuda")
    q[0, r, 0, 3 * r] = (1 + torch.rand(R, generator=g, device="cuda")).to(torch.bfloat16)
    k = torch.rand((n, D), generator=g, device="cuda").to(torch.bfloat16)
    scale = 1.0
    z = q[0, :, 0].double() @ k.double().T * scale
    p = torch.exp(z - z.amax(1, keepdim=True))                    # [R, n], the largest 1
    v = torch.randn((n, D), generator=g, device="cuda", dtype=torch.float64)
    v = (v - torch.linalg.pinv(p) @ (p @ v)).to(torch.bfloat16)
    kp, vp = (torch.zeros((pages, 1, ps, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kp[page, 0, j % ps], vp[page, 0, j % ps] = k, v
    c = dict(query=q, key_pages=kp, value_pages=vp, block_table=bt, page_size=ps,
             context_lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    out = decode(c, kind, False, scale=scale)[0, :, 0].double()
    check_no_device_error()
    l = p.sum(1, keepdim=True)
    want, mag = p @ v.double() / l, p @ v.double().abs() / l
    # scores: one exact product, scaled (2^-23 of at most 3) and into 2^x (2^-21)
    rest = 2.0 ** -16 + 2.0 ** -20 + n / 32 * 2.0 ** -24 + n / 64 * 2.0 ** -22
    tol = want.abs() * 2.0 ** -8 + mag * rest
    assert torch.all((out - want).abs() <= tol), float(((out - want).abs() / tol).max())
    # the bound would show a weight of one part
    once = p.to(torch.bfloat16).double() @ v.double() / l
    assert float(((once - want).abs() / tol).max()) > 3


@pytest.mark.parametrize("kind", ["window", "weights"])
@pytest.mark.parametrize("H_q,H_kv,L", [(8, 2, 1), (16, 1, 1), (5, 1, 3), (40, 1, 1), (8, 2, 8)])
@pytest.mark.parametrize("n", [300, 5000, 40000])
def test_e4m3_outputs_over_many_keys(kind, H_q, H_kv, L, n):
    c = make([n, n // 2 + 1], H_q, H_kv, L, 128, 16, seed=n + H_q, fp8=True)
    out = decode(c, kind, True).double()
    check_no_device_error()
    few = H_q // H_kv * L <= 16
    for b, m in enumerate(c["context_lens"].tolist()):
        j = torch.arange(m, device="cuda")
        page = c["block_table"][b, j // 16].long()
        for h in range(H_kv):
            k, v = (x[page, h, j % 16].view(F8).float().double() * s
                    for x, s in zip((c["key_pages"], c["value_pages"]), SCALES))
            q = c["query"][b].view(H_kv, -1, 128)[h].double()               # rows (head, i)
            z = q @ k.T / math.sqrt(128)
            i = torch.arange(len(q), device="cuda") % L
            z = z.masked_fill(j > (m - L + i)[:, None], -math.inf)
            p = torch.exp(z - z.amax(1, keepdim=True))
            l = p.sum(1, keepdim=True)
            want, mag = p @ v / l, p @ v.abs() / l
            size = float((q.abs() @ k.abs().T).max()) / math.sqrt(128)
            rest = 2.0 ** -11 * (1 if few else 2) + size * 2.0 ** -15 + m / 32 * 2.0 ** -24 + m / 64 * 2.0 ** -22
            tol = want.abs() * 2.0 ** -8 + mag * rest + 2.0 ** -25 * v.abs().sum(0) / l
            if not few:
                tol = tol + 2.0 ** -25 * SCALES[1]
            got = out[b].view(H_kv, -1, 128)[h]
            assert torch.all((got - want).abs() <= tol), float(((got - want).abs() / tol).max())
            # and the bound is well below what it bounds
            assert tol.square().mean() < (want.square().mean() / 25)
