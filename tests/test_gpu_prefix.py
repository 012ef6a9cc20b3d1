"""Decode behind shared prefixes against a plain 64-bit reference. Table entries of whole
prefix pages are -1 in the requests' own tables, and slots that no row sees hold NaN."""
import pytest
import torch

from gpu_util import check_no_device_error
from prefix_ref import check, make, reference
from window_ref import SCALES

pytestmark = pytest.mark.gpu


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


def call(c, kind="bf16", **kw):
    pa = _pa()
    f = {"bf16": pa.pa_decode_prefix, "e4m3": pa.pa_decode_prefix_fp8, "q4": pa.pa_decode_prefix_q4}[kind]
    scales = dict(k_scale=SCALES[0], v_scale=SCALES[1]) if kind == "e4m3" else {}
    return f(**c, **scales, **kw)


def run(prefixes, lens, H_q, H_kv, L, D, ps, seed, kind="bf16", **kw):
    c = make(prefixes, lens, H_q, H_kv, L, D, ps, seed, kind)
    out = call(c, kind, max_context_len=max(lens), **kw)
    check_no_device_error()
    check(out, reference(c, kind), kind, max(lens), 10.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("ps", [1, 4, 8, 16, 128, 256])
@pytest.mark.parametrize("plen", [1, 100, 128, 129, 700])
def test_one_prefix(plen, ps, kind):
    lens = [plen + x for x in (1, 0, 5, 64, 300, 2, 17)]
    run([(plen, 7)], lens, 8, 2, 1, 128, ps, seed=plen + ps, kind=kind)


@pytest.mark.parametrize("B", [1, 2, 16, 17, 32, 40, 80])
@pytest.mark.parametrize("H_q,H_kv", [(8, 1), (28, 4), (4, 4)])
def test_row_counts(H_q, H_kv, B):
    """One to several blocks of 256 rows, and up to 128 (both halves on the same rows)."""
    run([(500, B)], [500 + (37 * i) % 200 + 1 for i in range(B)], H_q, H_kv, 1, 128, 16, seed=B)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("L,H_q,H_kv", [(2, 4, 2), (4, 8, 1), (5, 7, 1), (17, 8, 2), (140, 2, 1)])
def test_several_rows(L, H_q, H_kv, kind):
    run([(333, 5)], [333 + x for x in (L, L + 1, 0, 400, 64)], H_q, H_kv, L, 128, 16, seed=L, kind=kind)


def test_head_dim_64():
    for ps in (2, 16, 64):
        run([(300, 9), (64, 3)], [300 + 7 * i for i in range(9)] + [65, 100, 64], 14, 2, 1, 64, ps, seed=ps)
    run([(1000, 40)], [1000 + i for i in range(40)], 8, 1, 2, 64, 16, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
def test_several_prefixes(kind):
    """Prefixes of none, of one request, of one tile and of many; requests without one."""
    prefixes = [(0, 3), (900, 1), (64, 20), (128, 0), (2500, 6), (77, 2)]
    lens = ([5, 0, 70] + [901] + [64 + 3 * i for i in range(20)] + [2500 + 100 * i for i in range(6)] + [77, 78] +
            [0, 1, 250])
    run(prefixes, lens, 8, 2, 1, 128, 16, seed=3, kind=kind)


def test_many_prefixes():
    prefixes = [(10 + 3 * i, 1 + i % 3) for i in range(150)]
    lens = [n + 1 + (7 * i) % 40 for i, (n, k) in enumerate(prefixes) for _ in range(k)]
    run(prefixes, lens, 4, 2, 1, 128, 16, seed=4)


def test_short_prefixes_beside_long_ones():
    """A block's share of the work is over 64 short prefixes (more than it lists in shared
    memory)."""
    prefixes = [(250000, 1), (250000, 1)] + [(5 + i % 3, 1) for i in range(100)]
    lens = [n + 1 + i % 5 for i, (n, _) in enumerate(prefixes)]
    run(prefixes, lens, 8, 8, 1, 64, 256, seed=13)


def test_requests_shorter_than_their_prefix():
    """Rows that see a part of the prefix, one key of it, or nothing."""
    run([(600, 8)], [600, 599, 300, 129, 128, 1, 0, 700], 8, 2, 1, 128, 16, seed=5)
    run([(600, 8)], [603, 601, 600, 130, 128, 2, 0, 700], 8, 2, 4, 128, 16, seed=6)


def test_long_prefix():
    run([(40000, 33)], [40000 + 50 * i for i in range(33)], 8, 1, 1, 128, 16, seed=7)


def test_tight_max_prefix_len_and_given_workspace():
    pa = _pa()
    c = make([(200, 4)], [201, 220, 300, 264], 8, 2, 1, 128, 16, seed=8)
    shape = pa.make_shape(c["query"].shape, c["key_pages"].shape, c["block_table"].shape[1])
    ws = torch.full((pa.pa_decode_prefix_workspace_bytes(shape, 16, 1, 200),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(c["query"], 3.0)
    for _ in range(2):                         # the second call finds the first one's states
        got = call(c, max_prefix_len=200, workspace=ws, out=out)
        assert got.data_ptr() == out.data_ptr()
        check_no_device_error()
        check(out, reference(c), "bf16", 300, 10.0)


def test_same_bits_twice_and_in_a_replayed_graph():
    for kind in ("bf16", "e4m3", "q4"):
        c = make([(1500, 20), (300, 3)], [1500 + 31 * i for i in range(20)] + [301, 400, 300], 8, 2, 1, 128, 16,
                 seed=9, pool=kind)
        want = call(c, kind)
        graph = torch.cuda.CUDAGraph()
        out = torch.empty_like(want)
        call(c, kind, out=out)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call(c, kind, out=out)
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)
        c["query"].mul_(0.5)
        graph.replay()
        assert torch.equal(out, call(c, kind)) and not torch.equal(out, want)


def test_other_stream():
    c = make([(700, 6)], [700 + 9 * i for i in range(6)], 8, 2, 1, 128, 16, seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = call(c, stream=side)
    side.synchronize()
    check(out, reference(c), "bf16", 745, 10.0)


def test_bad_values_are_recorded():
    pa = _pa()

    def flags(**bad):
        c = make([(300, 3), (200, 2)], [310, 300, 400, 200, 260], 4, 2, 1, 128, 16, seed=11, poison=False)
        for name, (at, value) in bad.items():
            c[name][at] = value
        call(c)
        st, got = pa.pa_get_device_error()
        assert st == pa.PA_ERR_DEVICE_BOUNDS, bad
        return got

    assert flags(prefix_table=((0, 3), 1 << 20)) == pa.PA_DEVERR_PAGE_ID
    assert flags(prefix_table=((1, 0), -1)) == pa.PA_DEVERR_PAGE_ID
    assert flags(block_table=((2, 20), 1 << 20)) == pa.PA_DEVERR_PAGE_ID
    assert flags(prefix_lens=(0, -4)) & pa.PA_DEVERR_CONTEXT_LEN
    assert flags(prefix_lens=(1, 10000)) & pa.PA_DEVERR_CONTEXT_LEN
    assert flags(context_lens=(1, 10000)) & pa.PA_DEVERR_CONTEXT_LEN
    for at, value in ((0, -1), (1, 9), (1, -7), (2, 6), (2, 2**31 - 1), (2, 1)):
        assert flags(prefix_starts=(at, value)) & pa.PA_DEVERR_PREFIX, (at, value)


def test_refusals():
    pa = _pa()
    c = make([(30, 2)], [40, 35], 4, 2, 1, 128, 16, seed=12)
    for bad in (dict(prefix_lens=c["prefix_lens"].repeat(2)), dict(prefix_starts=c["prefix_starts"][:1]),
                dict(prefix_table=c["prefix_table"][0]), dict(prefix_lens=c["prefix_lens"].cpu()),
                dict(query=c["query"][..., :64]), dict(page_size=8)):
        with pytest.raises(ValueError):
            call(dict(c, **bad))
    for bad in (dict(prefix_table=c["prefix_table"].long()), dict(prefix_starts=c["prefix_starts"].float()),
                dict(key_pages=c["key_pages"].half())):
        with pytest.raises(TypeError):
            call(dict(c, **bad))
    for kw in (dict(max_prefix_len=0), dict(max_prefix_len=-1), dict(scale=-1.0),
               dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(pa.PagedAttentionError):
            call(c, **kw)
    empty = dict(c, prefix_table=c["prefix_table"][:0], prefix_lens=c["prefix_lens"][:0],
                 prefix_starts=c["prefix_starts"][:1])
    with pytest.raises(pa.PagedAttentionError):
        call(empty)


def _limit(fits, hi=1 << 17):
    lo = 1
    while lo < hi:
        mid = (lo + hi + 1) // 2
        lo, hi = (mid, hi) if fits(mid) else (lo, mid - 1)
    return lo


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
def test_largest_batches(kind):
    """The largest batch that has a workspace runs; one more request is refused."""
    pa = _pa()
    need = {"bf16": pa.pa_decode_prefix_workspace_bytes, "e4m3": pa.pa_decode_prefix_fp8_workspace_bytes,
            "q4": pa.pa_decode_prefix_q4_workspace_bytes}[kind]
    n = _limit(lambda B: need(pa.pa_shape(B, 2, 1, 128, 1, 400, 3), 16, 2, 32) > 0)
    assert 2000 < n < 100000
    first, second = n // 2, n // 4
    lens = [20 + i % 9 for i in range(first)] + [32 + i % 7 for i in range(second)]
    lens += [i % 20 for i in range(n - len(lens))]
    c = make([(20, first), (32, second)], lens, 2, 1, 1, 128, 16, seed=3, pool=kind, poison=False)
    out = call(c, kind, max_context_len=48)
    check_no_device_error()
    some = torch.cat([torch.arange(8), first + torch.arange(8), n - 8 + torch.arange(8)]).cuda()
    part = dict(c, **{k: c[k][some] for k in ("query", "block_table", "context_lens")},
                prefix_starts=torch.tensor([0, 8, 16], dtype=torch.int32, device="cuda"))
    check(out[some], reference(part, kind), kind, 48, 10.0)
    more = dict(c, **{k: torch.cat([c[k], c[k][-1:]]) for k in ("query", "block_table", "context_lens")})
    with pytest.raises(pa.PagedAttentionError):
        call(more, kind)
