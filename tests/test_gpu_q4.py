"""4-bit page pools: the quantising append and the read-back bit by bit against numpy,
the attention over them against 64 bits."""
import numpy as np
import pytest
import torch

import q4_ref
from gpu_util import check_no_device_error
from q4_ref import D, ROW, dense_values, make, quantise, reference
from window_ref import check_out

pytestmark = pytest.mark.gpu


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def same_rows(got, want):
    """Rows with equal codes, and equal steps and least values (NaN is NaN, -0 is 0)."""
    assert np.array_equal(got[..., :64], want[..., :64])
    a, b = (np.ascontiguousarray(x[..., 64:]).view(np.float16) for x in (got, want))
    assert np.array_equal(a, b, equal_nan=True)


def special_rows(rng):
    """Rows [N, 128] bf16 at the borders: constants, ties, extremes, infinities, NaN."""
    x = rng.standard_normal((64, D)) * np.exp(rng.uniform(-12, 6, (64, 1)))
    x[0] = 0.0
    x[1] = -3.25
    x[2, :32] = np.arange(32) / 2                 # 15.5: step 1.033, quotients near halves
    x[3, :32] = np.arange(32) % 16                # step 1: codes themselves
    x[4, :32] = np.minimum(np.arange(32) / 2, 15) # step 1: ties at every other element
    x[5, :32] = -np.minimum(np.arange(32) / 2, 15)
    x[6] = 1e30
    x[7] = np.where(np.arange(D) % 2, 1e30, -1e30)
    x[8, 5] = np.inf
    x[9, 40] = -np.inf
    x[10, 70] = np.nan
    x[11] = np.where(np.arange(D) % 3, 2.0 ** -24, 2.0 ** -25)
    x[12] = rng.standard_normal(D) * 2.0 ** -24
    x[13] = rng.standard_normal(D) * 1e-30
    x[14] = 447 + rng.uniform(0, 4, D)
    x[15, ::32] = -448
    x[16, :] = -0.0
    x[17, :32] = 100 + np.arange(32) / 32
    return torch.from_numpy(x).to(torch.bfloat16)


def put(x_k, x_v, slots, P, H_kv, ps, fill=0xA5):
    pa = _pa()
    kp, vp = (torch.full((P, H_kv, ps, ROW), fill, dtype=torch.uint8, device="cuda") for _ in "kv")
    pa.pa_append_kv_q4(x_k.cuda(), x_v.cuda(), kp, vp, torch.tensor(slots, dtype=torch.int32, device="cuda"), ps)
    return kp, vp


@pytest.mark.parametrize("ps", [1, 4, 16, 256])
def test_append_is_exact(ps):
    rng = np.random.default_rng(ps)
    B, H_kv, L = 3, 2, 64
    rows = special_rows(rng)
    x_k = torch.randn(B, H_kv, L, D, generator=torch.Generator().manual_seed(ps)).to(torch.bfloat16)
    x_k[1, 1] = rows
    x_v = (x_k * 3).flip(-1).contiguous()
    P = 3 * (-(-L // ps)) + 2
    slots = rng.permutation(P * ps)[:B * L].reshape(B, L)
    slots[0, 5] = slots[2, 0] = -1
    kp, vp = put(x_k, x_v, slots.tolist(), P, H_kv, ps)
    check_no_device_error()
    for pool, x in ((kp, x_k), (vp, x_v)):
        got = pool.cpu().numpy()
        want = np.full_like(got, 0xA5)
        q = quantise(x.double().numpy())
        for b in range(B):
            for i in range(L):
                if slots[b, i] >= 0:
                    want[slots[b, i] // ps, :, slots[b, i] % ps] = q[b, :, i]
        same_rows(got, want)


def test_append_many_rows():
    """A million elements a scale: every code the nearest one."""
    for seed, std in ((1, 1.0), (2, 0.01), (3, 60.0)):
        g = torch.Generator().manual_seed(seed)
        x = (torch.randn(1, 4, 2048, D, generator=g) * std).to(torch.bfloat16)
        kp, vp = put(x, x.neg(), [list(range(2048))], 128, 4, 16)
        for pool, y in ((kp, x), (vp, x.neg())):
            got = pool.cpu().numpy().transpose(1, 0, 2, 3).reshape(4, 2048, ROW)
            same_rows(got, quantise(y[0].double().numpy()))


@pytest.mark.parametrize("ps", [1, 16, 128])
def test_read_back_is_exact(ps):
    pa = _pa()
    lens = [0, 1, 63, 64, 65, 200, 129]
    c = make(lens, 2, 2, 1, ps, seed=ps)
    dense_len = 200
    kd, vd = (torch.full((len(lens), 2, dense_len, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    got = pa.pa_gather_kv_q4(c["key_pages"], c["value_pages"], c["block_table"], c["context_lens"], ps, dense_len,
                             key_dense=kd, value_dense=vd)
    check_no_device_error()
    assert got[0] is kd or got[0].data_ptr() == kd.data_ptr()
    for dense, pool in ((kd, c["key_pages"]), (vd, c["value_pages"])):
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            rows = pool[c["block_table"][b, j // ps].long(), :, j % ps].transpose(0, 1).cpu().numpy()
            if n:
                assert np.array_equal(dense[b, :, :n].double().cpu().numpy(), dense_values(rows))
            assert torch.all(dense[b, :, n:] == 7.0)          # rows behind a context are left


def test_read_back_of_special_rows():
    pa = _pa()
    rows = special_rows(np.random.default_rng(0))[None, None]
    kp, vp = put(rows, rows, [list(range(64))], 4, 1, 16)
    bt = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    kd, vd = pa.pa_gather_kv_q4(kp, vp, bt, torch.tensor([64], dtype=torch.int32, device="cuda"), 16, 64)
    want = dense_values(quantise(rows[0].double().numpy()))
    for got in (kd, vd):
        assert np.array_equal(got[0].double().cpu().numpy(), want, equal_nan=True)


LENS = [0, 1, 2, 17, 31, 32, 33, 127, 128, 129, 300, 1000, 2500]


def check_decode(lens, H_q, H_kv, L, ps, seed, causal=True, mcl=True, std=1.0):
    c = make(lens, H_q, H_kv, L, ps, seed, std=std)
    out = _pa().pa_decode_q4(**c, causal=causal, max_context_len=max(lens) if mcl else 0)
    check_no_device_error()
    ref = reference(c, causal=causal)
    vmax = max(float(m.max()) for _, m, _, _ in ref)
    check_out(out, ref, True, max(lens), vmax)


@pytest.mark.parametrize("ps", [1, 2, 4, 8, 16, 32, 64, 256])
def test_one_row(ps):
    check_decode(LENS, 8, 2, 1, ps, seed=ps)


@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (7, 1), (28, 4), (8, 8), (16, 1), (33, 1)])
def test_head_layouts(H_q, H_kv):
    check_decode([5, 700, 90, 4100], H_q, H_kv, 1, 16, seed=H_q)


@pytest.mark.parametrize("L,H_q,H_kv", [(2, 4, 2), (5, 7, 1), (8, 8, 2), (16, 2, 1), (70, 4, 4)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_rows(L, H_q, H_kv, causal):
    check_decode(LENS, H_q, H_kv, L, 16, seed=L, causal=causal)


def test_unknown_max_context_len_and_many_requests():
    check_decode([(37 * i) % 900 for i in range(200)], 8, 8, 1, 16, seed=5, mcl=False)


def test_long_context():
    check_decode([40001, 3], 14, 2, 1, 64, seed=6)


def test_large_values():
    """Groups at the cut of 448 on both sides (-1024 s is still an f16)."""
    check_decode([100, 45], 4, 2, 1, 16, seed=7, std=150.0)


def test_large_queries_keep_the_least_values_exact():
    """Queries whose sum over a group is past f16's largest."""
    pa = _pa()
    c = make([64, 40], 4, 2, 1, 16, seed=8, std=2.0 ** -6)
    c["query"] = torch.full_like(c["query"], 4096.0)
    out = pa.pa_decode_q4(**c, scale=2.0 ** -9)
    check_out(out, reference(c, scale=2.0 ** -9), True, 64, 1.0)


@pytest.mark.parametrize("ps", [4, 16, 128])
@pytest.mark.parametrize("L,H_q,H_kv", [(9, 8, 2), (40, 7, 1), (130, 4, 4), (300, 8, 2)])
def test_prefill(L, H_q, H_kv, ps):
    pa = _pa()
    lens = [0, 5, L, L + 1, L + 127, 700]
    c = make(lens, H_q, H_kv, L, ps, seed=L)
    for f in (pa.pa_prefill_q4, pa.pa_attention_q4):
        out = f(**c, max_context_len=max(lens))
        check_no_device_error()
        check_out(out, reference(c, copied=True), False, max(lens))


@pytest.mark.parametrize("L,H_q,H_kv", [(300, 32, 8), (300, 28, 4), (700, 32, 8), (700, 28, 4)])
def test_prefill_of_many_rows(L, H_q, H_kv):
    """Enough (request, head pair, 128 rows) items for the kernel of pairs: even and odd groups,
    one to two items a block (tail pieces) and more."""
    pa = _pa()
    lens = [L, L + 1, 0, L - 200, L + 300, L + 129]
    c = make(lens, H_q, H_kv, L, 16, seed=L + H_q)
    out = pa.pa_attention_q4(**c, max_context_len=max(lens))
    check_no_device_error()
    check_out(out, reference(c, copied=True), False, max(lens))


@pytest.mark.parametrize("L", [1, 5, 40, 300])
def test_captured_calls_and_another_stream(L):
    """Attention and read-back in a graph on a stream of its own, replayed with other pools,
    queries, tables and lengths."""
    pa = _pa()
    lens, other = [L + 70, L, 333 + L, 0], [L + 5, L + 400, 0, L + 16]
    c, d = (make([n + 0 for n in x], 8, 2, L, 16, seed=L + i) for i, x in enumerate((lens, other)))
    P, W = (max(c[k].shape[i], d[k].shape[i]) for k, i in (("key_pages", 0), ("block_table", 1)))
    longest = max(lens + other)

    def padded(x):
        y = dict(x)
        for k in ("key_pages", "value_pages"):
            y[k] = torch.full((P, *x[k].shape[1:]), 0xFF, dtype=torch.uint8, device="cuda")
            y[k][:len(x[k])] = x[k]
        y["block_table"] = torch.full((len(lens), W), -1, dtype=torch.int32, device="cuda")
        y["block_table"][:, :x["block_table"].shape[1]] = x["block_table"]
        return y

    c, d = padded(c), padded(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pools = dict(key_pages=c["key_pages"], value_pages=c["value_pages"], block_table=c["block_table"],
                     context_lens=c["context_lens"], page_size=16, dense_len=longest)
        dense = [torch.zeros((4, 2, longest, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        out = pa.pa_attention_q4(**c, max_context_len=longest)
        pa.pa_gather_kv_q4(**pools, key_dense=dense[0], value_dense=dense[1])
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pa.pa_attention_q4(**c, max_context_len=longest, out=out)
            pa.pa_gather_kv_q4(**pools, key_dense=dense[0], value_dense=dense[1])
        for x in (c, d):
            want = pa.pa_attention_q4(**x, max_context_len=longest)
            for k in ("query", "key_pages", "value_pages", "block_table", "context_lens"):
                c[k].copy_(x[k])
            for t in dense:
                t.zero_()
            graph.replay()
            side.synchronize()
            assert torch.equal(out, want)
            check_out(out, reference(x, copied=L > 8), L <= 8, longest)
            for b, n in enumerate(x["context_lens"].tolist()):
                j = torch.arange(n, device="cuda")
                page = x["block_table"][b, j // 16].long()
                for t, pool in zip(dense, (x["key_pages"], x["value_pages"])):
                    rows = pool[page, :, j % 16].transpose(0, 1).cpu().numpy()
                    assert torch.equal(t[b, :, :n].cpu(), torch.from_numpy(dense_values(rows)).to(torch.bfloat16))
                    assert not t[b, :, n:].any()
    check_no_device_error()


def test_offsets_past_32_bits():
    """Rows whose byte offset in the pool is past 2^32."""
    pa = _pa()
    c = make([500], 4, 2, 1, 16, seed=9)
    used = c["key_pages"].shape[0]
    P = (1 << 32) // (2 * 16 * ROW) + 64
    for x in ("key_pages", "value_pages"):
        big = torch.full((P, 2, 16, ROW), 0xFF, dtype=torch.uint8, device="cuda")
        big[P - used:] = c[x]
        c[x] = big
    c["block_table"][c["block_table"] >= 0] += P - used
    out = pa.pa_decode_q4(**c)
    kd, _ = pa.pa_gather_kv_q4(c["key_pages"], c["value_pages"], c["block_table"], c["context_lens"], 16, 500)
    check_no_device_error()
    check_out(out, reference(c), True, 500, 10.0)
    j = torch.arange(500, device="cuda")
    rows = c["key_pages"][c["block_table"][0, j // 16].long(), :, j % 16].transpose(0, 1).cpu().numpy()
    assert np.array_equal(kd[0].double().cpu().numpy(), dense_values(rows))
    x = torch.randn(1, 2, 1, D, device="cuda").to(torch.bfloat16)
    pa.pa_append_kv_q4(x, x, c["key_pages"], c["value_pages"],
                       torch.tensor([[P * 16 - 1]], dtype=torch.int32, device="cuda"), 16)
    same_rows(c["key_pages"][P - 1, :, 15].cpu().numpy(), quantise(x[0, :, 0].double().cpu().numpy()))


def test_bad_slots_pages_and_lengths_are_recorded():
    pa = _pa()
    x = torch.randn(1, 2, 3, D, device="cuda").to(torch.bfloat16)
    kp, vp = (torch.zeros((4, 2, 16, ROW), dtype=torch.uint8, device="cuda") for _ in "kv")
    pa.pa_append_kv_q4(x, x, kp, vp, torch.tensor([[-5, 64, 1 << 30]], dtype=torch.int32, device="cuda"), 16)
    assert pa.pa_get_device_error() == (pa.PA_ERR_DEVICE_BOUNDS, pa.PA_DEVERR_SLOT)
    assert not kp.any() and not vp.any()
    for what in ("decode", "prefill", "gather"):
        for field, at, bad, flag in (("block_table", (0, 300 // 16), 1 << 20, pa.PA_DEVERR_PAGE_ID),
                                     ("block_table", (0, 2), -1, pa.PA_DEVERR_PAGE_ID),
                                     ("context_lens", (1,), 1000, pa.PA_DEVERR_CONTEXT_LEN),
                                     ("context_lens", (1,), -1, pa.PA_DEVERR_CONTEXT_LEN)):
            c = make([300, 200], 4, 2, 1, 16, seed=8, poison=False)
            c[field][at] = bad
            if what == "gather":
                pa.pa_gather_kv_q4(c["key_pages"], c["value_pages"], c["block_table"], c["context_lens"], 16, 300)
            elif what == "decode":
                pa.pa_decode_q4(**c)
            else:
                pa.pa_prefill_q4(**c, max_context_len=300)
            st, flags = pa.pa_get_device_error()
            # a context past its table row reads entries of -1 too
            assert st == pa.PA_ERR_DEVICE_BOUNDS and flags & flag, (what, field, bad)


def test_refusals():
    pa = _pa()
    c = make([30, 20], 4, 2, 1, 16, seed=9)
    x = torch.zeros(2, 2, 1, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for bad in (dict(query=c["query"][..., :64]), dict(key_pages=c["key_pages"][..., :64]),
                dict(page_size=8), dict(context_lens=c["context_lens"][:1]), dict(query=c["query"].cpu()),
                dict(workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            pa.pa_decode_q4(**dict(c, **bad))
    for bad in (dict(query=c["query"].float()), dict(key_pages=c["key_pages"].view(torch.int8)),
                dict(block_table=c["block_table"].long())):
        with pytest.raises(TypeError):
            pa.pa_decode_q4(**dict(c, **bad))
    for f, kw in ((pa.pa_decode_q4, {}), (pa.pa_prefill_q4, dict(max_context_len=30))):
        with pytest.raises(pa.PagedAttentionError):
            f(**c, **kw, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        with pytest.raises(pa.PagedAttentionError):
            f(**c, **kw, scale=0.0)
    with pytest.raises(ValueError):
        pa.pa_append_kv_q4(x, x, c["key_pages"], c["value_pages"], slots[:1], 16)
    with pytest.raises(ValueError):
        pa.pa_append_kv_q4(x[..., :64], x[..., :64], c["key_pages"], c["value_pages"], slots, 16)
    with pytest.raises(ValueError):
        pa.pa_append_kv_q4(x, x, c["key_pages"].expand(-1, -1, -1, ROW)[..., :64], c["value_pages"], slots, 16)
    with pytest.raises(ValueError):
        pa.pa_gather_kv_q4(c["key_pages"], c["value_pages"], c["block_table"], c["context_lens"], 16, 30,
                           key_dense=torch.zeros(2, 2, 29, D, dtype=torch.bfloat16, device="cuda"))
    assert q4_ref.ROW == c["key_pages"].shape[3]


def test_empty_calls():
    pa = _pa()
    kp, vp = (torch.zeros((4, 2, 16, ROW), dtype=torch.uint8, device="cuda") for _ in "kv")
    none = torch.zeros(2, 2, 0, D, dtype=torch.bfloat16, device="cuda")
    pa.pa_append_kv_q4(none, none, kp, vp, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), 16)
    kd, vd = pa.pa_gather_kv_q4(kp, vp, torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                                torch.zeros(0, dtype=torch.int32, device="cuda"), 16, 5)
    assert kd.shape == (0, 2, 5, D) == vd.shape


def test_largest_batch():
    """The largest batch that has a workspace runs; one more request is refused."""
    pa = _pa()
    fits = lambda B: pa.pa_decode_q4_workspace_bytes(pa.pa_shape(B, 2, 1, D, 1, 400, 3)) > 0  # noqa: E731
    lo, hi = 1, 1 << 17
    while lo < hi:
        mid = (lo + hi + 1) // 2
        lo, hi = (mid, hi) if fits(mid) else (lo, mid - 1)
    assert 2000 < lo < 100000
    lens = [i % 37 for i in range(lo)]
    c = make(lens, 2, 1, 1, 16, seed=11, poison=False)
    out = pa.pa_attention_q4(**c, max_context_len=36)
    check_no_device_error()
    some = torch.cat([torch.arange(40), lo - 40 + torch.arange(40)]).cuda()
    part = dict(c, **{k: c[k][some] for k in ("query", "block_table", "context_lens")})
    check_out(out[some], reference(part), True, 36)
    more = dict(c, **{k: torch.cat([c[k], c[k][-1:]]) for k in ("query", "block_table", "context_lens")})
    with pytest.raises(pa.PagedAttentionError):
        pa.pa_attention_q4(**more, max_context_len=36)
