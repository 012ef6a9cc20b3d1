"""pa_kv_evict against a plain implementation: which positions are kept, and
every byte of the pools afterwards. Positions are whole numbers and rows are
copied, so nothing has a tolerance."""
import numpy as np
import pytest
import torch

from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def make(lens, H_kv, D, ps, keep, seed, fp8=False, dst="same", weights="spread", max_pages=None):
    rng = np.random.default_rng(seed)
    B = len(lens)
    counts = [-(-n // ps) for n in lens]
    width = max_pages or max(max(counts), 1)
    dcount = [-(-min(n, keep) // ps) for n in lens]
    P = sum(counts) + sum(dcount) + 5
    perm = rng.permutation(P).astype(np.int32)
    bt = np.full((B, width), -1, np.int32)
    at = 0
    for b, k in enumerate(counts):
        bt[b, :k] = perm[at:at + k]
        at += k
    if dst == "same":
        dt = bt
    else:
        dt = np.full((B, max(max(dcount), -(-min(keep, width * ps) // ps), 1)), 1 << 20, np.int32)
        for b, k in enumerate(dcount):
            dt[b, :k] = perm[at:at + k]
            at += k
    shape = (P, H_kv, ps, D)
    if fp8:
        k, v = (rng.integers(0, 256, shape).astype(np.uint8) for _ in "kv")
    else:
        k, v = (rng.integers(-32768, 32768, shape).astype(np.int16) for _ in "kv")
    w = (rng.random((P, H_kv, ps)) ** 6).astype(np.float32)
    if weights == "ties":
        w = np.round(w * 3).astype(np.float32)
    elif weights == "odd":                # NaN, infinities, zeros of both signs, negatives
        odd = np.float32([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1.0, -np.nan])
        w = np.where(rng.random(w.shape) < 0.6, odd[rng.integers(0, 8, w.shape)], w)
    elif weights == "same":
        w[:] = 0.25
    return dict(k=k, v=v, w=w, bt=bt, dt=dt, cl=np.int32(lens), ps=ps, fp8=fp8)


def plain(c, keep, S, R):
    """(kept, new_lens, pools) by sorting the positions of each (request, head)."""
    B, H = len(c["cl"]), c["k"].shape[1]
    kept = np.full((B, H, keep), -1, np.int32)
    new = np.minimum(c["cl"], keep).astype(np.int32)
    pools = [c[x].copy() for x in "kvw"]
    ps = c["ps"]
    for b, n in enumerate(c["cl"]):
        pos = np.arange(n)
        page, off = c["bt"][b, pos // ps], pos % ps
        for h in range(H):
            w = c["w"][page, h, off].astype(np.float64)
            order = [(1 if np.isnan(x) else 0, -x if not np.isnan(x) else 0.0, p) for p, x in zip(pos, w)]
            if n <= keep:
                mine = pos
            else:
                between = sorted(order[S:n - R])[:keep - S - R]
                mine = np.concatenate([pos[:S], np.sort(np.int64([t[2] for t in between])), pos[n - R:]])
            mine = mine.astype(np.int64)
            kept[b, h, :len(mine)] = mine
            to = np.arange(len(mine))
            for i, x in enumerate("kvw"):
                pools[i][c["dt"][b, to // ps], h, to % ps] = c[x][page[mine], h, off[mine]]
    return kept, new, pools


def device(c):
    def pool(x):
        t = torch.from_numpy(x).cuda()
        return t if c["fp8"] else t.view(torch.bfloat16)
    d = dict(key_pages=pool(c["k"]), value_pages=pool(c["v"]),
             weight_pages=torch.from_numpy(c["w"]).cuda(), block_table=torch.from_numpy(c["bt"]).cuda(),
             context_lens=torch.from_numpy(c["cl"]).cuda(), page_size=c["ps"])
    d["dst_block_table"] = None if c["dt"] is c["bt"] else torch.from_numpy(c["dt"]).cuda()
    return d


def same_bits(t, x):
    t = t.cpu()
    t = t.view(torch.int16) if t.dtype == torch.bfloat16 else t
    got, x = np.ascontiguousarray(t.numpy()), np.ascontiguousarray(x)
    return np.array_equal(got.view(np.uint8), x.view(np.uint8))


def check(c, keep, S=0, R=0):
    pa = _pa()
    d = device(c)
    f = pa.pa_kv_evict_fp8 if c["fp8"] else pa.pa_kv_evict
    kept, new = f(**d, keep=keep, sinks=S, recent=R)
    check_no_device_error()
    want_kept, want_new, pools = plain(c, keep, S, R)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(new.cpu().numpy(), want_new)
    for t, x in zip((d["key_pages"], d["value_pages"], d["weight_pages"]), pools):
        assert same_bits(t, x)


LENS = [0, 1, 7, 63, 64, 65, 200, 201, 1030, 1500]


@pytest.mark.parametrize("dst", ["same", "other"])
@pytest.mark.parametrize("ps", [1, 4, 16, 256])
@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (128, True)])
def test_matches_the_definition(D, fp8, ps, dst):
    check(make(LENS, 2, D, ps, 64, seed=ps + D, fp8=fp8, dst=dst), 64, 4, 10)


@pytest.mark.parametrize("keep,S,R", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (10, 5, 5), (200, 0, 0),
                                      (200, 0, 199), (200, 200, 0), (201, 3, 0), (1029, 4, 64),
                                      (1030, 4, 64), (1500, 1, 1), (4000, 4, 100)])
@pytest.mark.parametrize("dst", ["same", "other"])
def test_budgets(keep, S, R, dst):
    check(make(LENS, 3, 128, 16, keep, seed=keep + S, dst=dst), keep, S, R)


@pytest.mark.parametrize("weights", ["ties", "odd", "same"])
@pytest.mark.parametrize("keep,S,R", [(40, 0, 0), (170, 4, 32)])
def test_ties_and_special_weights(weights, keep, S, R):
    check(make(LENS + [2300], 2, 64, 8, keep, seed=9, weights=weights), keep, S, R)


@pytest.mark.parametrize("n,keep", [(4097, 4096), (33000, 8192), (70001, 35000)])
def test_long_contexts(n, keep):
    check(make([n, n // 3], 2, 64, 16, keep, seed=n, weights="spread"), keep, 4, 128)


def test_many_requests():
    rng = np.random.default_rng(4)
    check(make([int(x) for x in rng.integers(0, 400, 130)], 8, 64, 32, 100, seed=4), 100, 2, 20)


def test_pages_shared_by_requests_go_to_fresh_ones():
    c = make([300, 300, 150], 2, 128, 16, 128, seed=12, dst="other")
    c["bt"][1, :10] = c["bt"][0, :10]
    check(c, 128, 4, 16)


def test_bad_lengths_and_pages_are_recorded():
    pa = _pa()
    c = make([200, 90, 64], 2, 64, 16, 50, seed=13, dst="other")
    d = device(c)
    d["context_lens"][1] = -3
    kept, new = pa.pa_kv_evict(**d, keep=50)
    assert pa.pa_get_device_error() == (pa.PA_ERR_DEVICE_BOUNDS, pa.PA_DEVERR_CONTEXT_LEN)
    assert new.tolist() == [50, 0, 50] and torch.all(kept[1] == -1)
    d = device(c)
    before = [d[x].clone() for x in ("key_pages", "value_pages", "weight_pages")]
    d["block_table"][0, 2] = 1 << 24
    d["dst_block_table"][2, 1] = -7
    kept, new = pa.pa_kv_evict(**d, keep=50, sinks=40)
    assert pa.pa_get_device_error() == (pa.PA_ERR_DEVICE_BOUNDS, pa.PA_DEVERR_PAGE_ID)
    # positions 32..39 of request 0 stay chosen (sinks) and are not moved
    assert kept[0, 0, :40].tolist() == list(range(40))
    page = int(d["dst_block_table"][0, 2])
    for old, t in zip(before, (d["key_pages"], d["value_pages"], d["weight_pages"])):
        a, b = (x[page, :, :8].contiguous().view(torch.uint8) for x in (old, t))
        assert torch.equal(a, b)


def test_own_page_in_another_table_is_recorded_and_not_written():
    pa = _pa()
    c = make([200], 2, 64, 16, 64, seed=17, dst="other")
    d = device(c)
    before = d["key_pages"].clone()
    d["dst_block_table"][0, 1] = d["block_table"][0, 1]
    kept, _ = pa.pa_kv_evict(**d, keep=64)
    assert pa.pa_get_device_error() == (pa.PA_ERR_DEVICE_BOUNDS, pa.PA_DEVERR_PAGE_ID)
    want, _, _ = plain(c, 64, 0, 0)
    assert np.array_equal(kept.cpu().numpy(), want)
    page = int(d["block_table"][0, 1])
    assert torch.equal(before[page].view(torch.int16), d["key_pages"][page].view(torch.int16))


def test_offsets_past_32_bits():
    """Rows whose byte offset is past 2^32 move; nothing else does."""
    pa = _pa()
    P, H, ps, D = (1 << 24) // (16 * 2) + 40, 2, 16, 128          # 2^24 rows of 256 bytes
    k = torch.zeros((P, H, ps, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    w = torch.zeros((P, H, ps), device="cuda")
    bt = torch.arange(P - 30, P - 10, dtype=torch.int32, device="cuda").view(1, 20)
    dt = torch.arange(P - 10, P, dtype=torch.int32, device="cuda").view(1, 10)
    g = torch.Generator(device="cuda").manual_seed(1)
    k[P - 30:P - 10] = torch.randn((20, H, ps, D), generator=g, device="cuda").to(torch.bfloat16)
    v[P - 30:P - 10] = torch.randn((20, H, ps, D), generator=g, device="cuda").to(torch.bfloat16)
    w[P - 30:P - 10] = torch.rand((20, H, ps), generator=g, device="cuda")
    kept, _ = pa.pa_kv_evict(k, v, w, bt, torch.tensor([320], dtype=torch.int32, device="cuda"), 16,
                             160, 4, 8, dt)
    check_no_device_error()
    for h in range(H):
        p = kept[0, h].long()
        for pool in (k, v, w):
            src = pool[P - 30:P - 10, h].reshape(320, -1)[p]
            assert torch.equal(pool[P - 10:, h].reshape(160, -1), src)
    assert int((k[:P - 30] != 0).sum()) == 0 and int((w[:P - 30] != 0).sum()) == 0


def test_python_refusals():
    pa = _pa()
    d = device(make([100, 90], 2, 64, 16, 50, seed=14))
    for bad, err in ((dict(keep=0), pa.PagedAttentionError), (dict(sinks=30, recent=30), pa.PagedAttentionError),
                     (dict(page_size=8), ValueError), (dict(weight_pages=d["weight_pages"].double()), TypeError),
                     (dict(weight_pages=d["weight_pages"][:, :1]), ValueError),
                     (dict(block_table=d["block_table"].long()), TypeError),
                     (dict(context_lens=d["context_lens"][:1]), ValueError),
                     (dict(context_lens=d["context_lens"].cpu()), ValueError),
                     (dict(dst_block_table=d["block_table"][:, :2].contiguous()), pa.PagedAttentionError),
                     (dict(new_lens=d["context_lens"]), pa.PagedAttentionError),
                     (dict(kept=torch.empty((2, 2, 49), dtype=torch.int32, device="cuda")), ValueError)):
        before = d["key_pages"].clone()
        with pytest.raises(err):
            pa.pa_kv_evict(**{**dict(d, keep=50), **bad})
        torch.cuda.synchronize()
        assert torch.equal(before.view(torch.int16), d["key_pages"].view(torch.int16))


def test_other_stream_and_replayed_graph():
    pa = _pa()
    c = make([500, 333], 2, 128, 16, 128, seed=15, dst="other")
    want_kept, want_new, pools = plain(c, 128, 4, 16)
    d = device(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kept, new = pa.pa_kv_evict(**d, keep=128, sinks=4, recent=16, stream=side)
    side.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert same_bits(d["key_pages"], pools[0])
    d = device(c)
    kept, new = torch.zeros_like(kept), torch.zeros_like(new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_kv_evict(**d, keep=128, sinks=4, recent=16, kept=kept, new_lens=new)
    fresh = make([500, 333], 2, 128, 16, 128, seed=16, dst="other")
    for t, x in ((d["key_pages"], "k"), (d["value_pages"], "v")):
        t.view(torch.int16).copy_(torch.from_numpy(fresh[x]))
    d["weight_pages"].copy_(torch.from_numpy(fresh["w"]))
    d["block_table"].copy_(torch.from_numpy(fresh["bt"]))
    d["dst_block_table"].copy_(torch.from_numpy(fresh["dt"]))
    graph.replay()
    torch.cuda.synchronize()
    want_kept, _, pools = plain(fresh, 128, 4, 16)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert same_bits(d["key_pages"], pools[0]) and same_bits(d["value_pages"], pools[1])
