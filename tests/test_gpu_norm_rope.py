"""pa_qk_norm_rope_append against a plain implementation in 64 bits.

Tolerance, per element: the result is rounded once, to bf16 (half a step,
2^-8 relative) or to an e4m3 code (2^-4 relative, or half the smallest
subnormal step, 2^-10 of the scale). The fp32 work before it: the mean of D
squares (D + 4 roundings of 2^-24 at most, halved by the root), the inverse
root (2 ulp), two products, and a rotation whose two terms are each below
|x| + |x'| in size: below 2^-17 * (|x| + |x'|) for D <= 128 (128/2 + 10
roundings of 2^-24). A term this small can still move a value across a
rounding border, which costs one full step; hence bf16 outputs may be off by
2^-8 |ref| + 2^-17 (|x| + |x'|), the sum of both.
"""
import numpy as np
import pytest
import torch

from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def make(B, L, H_q, H_kv, D, ps, R, seed, norm=(True, True), std=1.5, table=4096, fp8=False,
         row_pad=0, batch_pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = (H_q + 2 * H_kv) * D
    big = torch.randn((B, L + batch_pad, width + row_pad), generator=g, device="cuda") * std
    qkv = big.to(torch.bfloat16)[:, :L, :width]
    P = (B * L + ps - 1) // ps + 3
    slots = torch.randperm(P * ps, generator=g, device="cuda")[:B * L].view(B, L).to(torch.int32)
    angle = torch.arange(table, device="cuda", dtype=torch.float64)[:, None] * \
        (10000.0 ** (-torch.arange(0, max(R, 2), 2, device="cuda", dtype=torch.float64) / max(R, 2)))
    shape = (P, H_kv, ps, D)
    if fp8:
        pools = [torch.randint(0, 127, shape, generator=g, device="cuda").to(torch.uint8) for _ in "kv"]
    else:
        pools = [torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
    weights = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) if w else None
               for w in norm]
    return dict(qkv=qkv, q_weight=weights[0], k_weight=weights[1],
                cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float() if R else None,
                positions=torch.randint(0, table, (B, L), generator=g, device="cuda").to(torch.int32),
                key_pages=pools[0], value_pages=pools[1], slot_mapping=slots, page_size=ps)


def plain(c, inter):
    """(queries [B, H_q, L, D], keys and values [B, L, H_kv, D], sizes) in 64 bits."""
    P, H_kv, ps, D = c["key_pages"].shape
    B, L, width = c["qkv"].shape
    H_q = width // D - 2 * H_kv
    x = c["qkv"].double().reshape(B, L, -1, D)
    parts, sizes = [], []
    for y, w in ((x[:, :, :H_q], c["q_weight"]), (x[:, :, H_q:H_q + H_kv], c["k_weight"])):
        if w is not None:
            y = y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + EPS) * w.double()
        size = y.abs()
        if c["cos_sin"] is not None:
            R = c["cos_sin"].shape[1]
            t = c["cos_sin"].double()[c["positions"].long().clamp(0, c["cos_sin"].shape[0] - 1)]
            co, si = t[..., :R // 2].unsqueeze(2), t[..., R // 2:].unsqueeze(2)
            y, size = y.clone(), size.clone()
            lo, hi = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
            p, q = y[..., lo].clone(), y[..., hi].clone()
            y[..., lo], y[..., hi] = p * co - q * si, q * co + p * si
            size[..., lo] = size[..., hi] = p.abs() + q.abs()
        parts.append(y)
        sizes.append(size)
    return parts[0].transpose(1, 2), parts[1], x[:, :, H_q + H_kv:], sizes[0].transpose(1, 2), sizes[1]


def check(c, query, before, inter, scales=None):
    q, k, v, qs, ks = plain(c, inter)
    ps = c["page_size"]
    assert torch.all((query.double() - q).abs() <= q.abs() * 2.0 ** -8 + qs * 2.0 ** -17 + 1e-38)
    slot = c["slot_mapping"].long()
    ok = slot >= 0
    page, off = slot[ok] // ps, slot[ok] % ps
    for i, (pool, old, ref, size) in enumerate(((c["key_pages"], before[0], k, ks),
                                                (c["value_pages"], before[1], v, v.abs()))):
        got = pool[page, :, off]
        want = ref[ok]
        if scales is None:
            if i == 1:
                assert torch.equal(got.double(), want)
            tol = want.abs() * 2.0 ** -8 + size[ok] * 2.0 ** -17 + 1e-38
            assert torch.all((got.double() - want).abs() <= tol)
        else:
            val = got.view(torch.float8_e4m3fn).float().double()
            want = (want / scales[i]).clamp(-448, 448)
            tol = want.abs() * 2.0 ** -4 + 2.0 ** -10 + size[ok] / scales[i] * 2.0 ** -17
            assert torch.all((val - want).abs() <= tol)
        # every other slot is as it was
        mine = torch.zeros(pool.shape[0], ps, dtype=torch.bool, device="cuda")
        mine[page, off] = True
        assert torch.equal(pool.transpose(1, 2)[~mine], old.transpose(1, 2)[~mine])


def run(c, inter=False, scales=None, **kw):
    pa = _pa()
    before = c["key_pages"].clone(), c["value_pages"].clone()
    f = pa.pa_qk_norm_rope_append if scales is None else pa.pa_qk_norm_rope_append_fp8
    named = dict(c)
    if scales is not None:
        named.update(k_scale=scales[0], v_scale=scales[1])
    query = f(**named, eps=EPS, interleaved=inter, **kw)
    return query, before


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,L,H_q,H_kv,D,ps,R", [
    (1, 1, 28, 4, 128, 16, 128), (1, 1, 1, 1, 64, 1, 64), (3, 5, 8, 8, 64, 4, 32),
    (2, 37, 7, 1, 128, 128, 64), (5, 3, 4, 2, 128, 256, 16), (1, 700, 32, 8, 128, 16, 128),
    (2, 33, 6, 2, 128, 2, 96), (2, 40, 4, 2, 64, 8, 48), (2, 9, 4, 4, 128, 16, 0),
    (64, 1, 32, 8, 128, 64, 128)])
def test_matches_the_formula(B, L, H_q, H_kv, D, ps, R, inter):
    c = make(B, L, H_q, H_kv, D, ps, R, seed=B * 100 + L + R)
    query, before = run(c, inter)
    check_no_device_error()
    check(c, query, before, inter)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,L,H_q,H_kv,ps,R", [(1, 1, 28, 4, 16, 128), (3, 21, 8, 2, 4, 64),
                                               (2, 300, 32, 8, 128, 128)])
def test_e4m3_pools(B, L, H_q, H_kv, ps, R, inter):
    c = make(B, L, H_q, H_kv, 128, ps, R, seed=L, fp8=True)
    query, before = run(c, inter, scales=(0.02, 0.05))
    check_no_device_error()
    check(c, query, before, inter, scales=(0.02, 0.05))


def test_e4m3_codes_are_those_of_the_plain_append():
    """Without norm and rotation the rows are pa_append_kv_fp8's, saturation and
    NaN included."""
    pa = _pa()
    c = make(2, 19, 4, 2, 128, 16, 0, seed=3, norm=(False, False), fp8=True)
    c["qkv"][0, 0, 4 * 128:4 * 128 + 6] = torch.tensor([600., -600., 1e-6, 0., float("nan"), 20.])
    kp, vp = c["key_pages"].clone(), c["value_pages"].clone()
    run(c, scales=(0.05, 0.03))
    x = c["qkv"].view(2, 19, 8, 128).transpose(1, 2)
    pa.pa_append_kv_fp8(x[:, 4:6].contiguous(), x[:, 6:8].contiguous(), kp, vp, c["slot_mapping"], 16,
                        0.05, 0.03)
    assert torch.equal(c["key_pages"], kp) and torch.equal(c["value_pages"], vp)


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
def test_norm_of_either_side_alone(norm):
    c = make(2, 13, 6, 2, 128, 16, 128, seed=5, norm=norm)
    query, before = run(c)
    check(c, query, before, False)


@pytest.mark.parametrize("D", [64, 128])
def test_strided_rows(D):
    """Rows inside a wider projection, batches further apart than L rows."""
    c = make(3, 6, 4, 2, D, 16, D, seed=6, row_pad=24, batch_pad=2)
    assert not c["qkv"].is_contiguous()
    query, before = run(c)
    check(c, query, before, False)


def test_padding_tokens_and_bad_values():
    pa = _pa()
    c = make(2, 6, 4, 2, 128, 16, 128, seed=7, table=50)
    c["slot_mapping"][0, :2] = -1
    c["positions"][0, 0] = 1 << 30          # padding: clamped, not recorded
    c["positions"][0, 1] = -5
    query, before = run(c)
    check_no_device_error()
    check(c, query, before, False)
    c["positions"][1, 3] = 50               # a token behind the table
    query, before = run(c)
    st, flags = pa.pa_get_device_error()
    assert st == pa.PA_ERR_DEVICE_BOUNDS and flags == pa.PA_DEVERR_POSITION
    c["positions"][1, 3] = 49
    c["slot_mapping"][1, 4] = c["key_pages"].shape[0] * 16
    before = c["key_pages"].clone(), c["value_pages"].clone()
    query, _ = run(c)
    st, flags = pa.pa_get_device_error()
    assert st == pa.PA_ERR_DEVICE_BOUNDS and flags == pa.PA_DEVERR_SLOT
    c["slot_mapping"][1, 4] = -1
    check(c, query, before, False)


def test_zero_rows_norm_to_zero():
    c = make(1, 3, 4, 2, 128, 16, 128, seed=8)
    c["qkv"][0, 1] = 0
    query, before = run(c)
    check(c, query, before, False)
    assert torch.all(query[0, :, 1] == 0)


def test_no_tokens_touch_nothing():
    c = make(1, 1, 4, 2, 128, 16, 128, seed=9)
    c["qkv"], c["positions"] = c["qkv"][:, :0], c["positions"][:, :0].contiguous()
    c["slot_mapping"] = c["slot_mapping"][:, :0].contiguous()
    query, before = run(c)
    assert query.shape == (1, 4, 0, 128)
    assert torch.equal(c["key_pages"], before[0])


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: the last slot is written, its mirror
    2^32 bytes (2^31 elements) before is not."""
    P, ps, H_kv, D = (1 << 31) // (16 * 2 * 128) + 8, 16, 2, 128
    c = make(1, 2, 4, 2, 128, 16, 128, seed=10)
    c["key_pages"] = torch.zeros((P, H_kv, ps, D), dtype=torch.bfloat16, device="cuda")
    c["value_pages"] = torch.zeros_like(c["key_pages"])
    c["slot_mapping"] = torch.tensor([[P * ps - 1, P * ps - 20]], dtype=torch.int32, device="cuda")
    _pa().pa_qk_norm_rope_append(**c, eps=EPS)
    check_no_device_error()
    _, k, v, _, ks = plain(c, False)
    for t, slot in enumerate((P * ps - 1, P * ps - 20)):
        assert torch.equal(c["value_pages"][slot // ps, :, slot % ps].double(), v[0, t])
    assert int((c["value_pages"].view(-1, 128)[:1 << 16] != 0).sum()) == 0


def test_python_refusals():
    pa = _pa()
    c = make(2, 3, 4, 2, 128, 16, 128, seed=11)
    for bad, err in ((dict(qkv=c["qkv"].float()), TypeError), (dict(qkv=c["qkv"].cpu()), ValueError),
                     (dict(qkv=c["qkv"][..., :-128]), pa.PagedAttentionError),
                     (dict(qkv=c["qkv"][..., :-8]), ValueError),
                     (dict(q_weight=c["q_weight"][:64]), ValueError),
                     (dict(positions=c["positions"][:1]), ValueError),
                     (dict(positions=c["positions"].long()), TypeError),
                     (dict(slot_mapping=c["slot_mapping"][:, :2]), ValueError),
                     (dict(page_size=8), ValueError),
                     (dict(key_pages=c["key_pages"].cpu()), ValueError),
                     (dict(cos_sin=c["cos_sin"][:, :40].contiguous()), pa.PagedAttentionError)):
        before = c["key_pages"].clone()
        with pytest.raises(err):
            pa.pa_qk_norm_rope_append(**dict(c, **bad))
        assert torch.equal(before, c["key_pages"])
    with pytest.raises(pa.PagedAttentionError):   # queries over the projection's own memory
        pa.pa_qk_norm_rope_append(**c, query=c["qkv"].reshape(-1)[:2 * 4 * 3 * 128].view(2, 4, 3, 128))


def test_other_stream_and_replayed_graph():
    pa = _pa()
    c = make(2, 5, 8, 2, 128, 16, 128, seed=12)
    want, _ = run(c)
    kp = c["key_pages"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c["key_pages"].zero_()
    torch.cuda.synchronize()
    got = pa.pa_qk_norm_rope_append(**c, eps=EPS, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_qk_norm_rope_append(**c, eps=EPS, query=out)
    c["qkv"].mul_(2)
    c["positions"].fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    q, k, v, qs, ks = plain(c, False)
    assert torch.all((out.double() - q).abs() <= q.abs() * 2.0 ** -8 + qs * 2.0 ** -17)
