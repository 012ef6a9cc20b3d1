"""Calls at the edges of what the 4-bit pages and the decode behind shared prefixes document:
requests before the first prefix and between prefixes, as many prefixes as there may be, pools
past 32 bits, appends of more rows than a launch has blocks, calls from several host threads."""
import threading

import pytest
import torch

from gpu_util import check_no_device_error
from prefix_ref import check, make, reference
from q4_ref import ROW

pytestmark = pytest.mark.gpu


def call(c, kind="bf16", **kw):
    import paged_kv_attention_06_gb300 as pa
    from window_ref import SCALES
    f = {"bf16": pa.pa_decode_prefix, "e4m3": pa.pa_decode_prefix_fp8, "q4": pa.pa_decode_prefix_q4}[kind]
    return f(**c, **(dict(k_scale=SCALES[0], v_scale=SCALES[1]) if kind == "e4m3" else {}), **kw)


def moved(c, order):
    """The same requests in another order."""
    at = torch.tensor(order, device="cuda")
    return dict(c, **{k: c[k][at].contiguous() for k in ("query", "block_table", "context_lens")})


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
def test_requests_before_the_first_prefix(kind):
    """starts 3, 7, 7, 12 of 15 requests: three without a prefix in front, three behind."""
    lens = [310 + i for i in range(4)] + [140 + 50 * i for i in range(5)] + [60, 0, 33, 1, 500, 16]
    c = make([(300, 4), (77, 0), (128, 5)], lens, 8, 2, 1, 128, 16, seed=1, pool=kind)
    c = moved(c, [9, 10, 11, *range(9), 12, 13, 14])
    c["prefix_starts"] += 3
    out = call(c, kind)
    check_no_device_error()
    check(out, reference(c, kind), kind, 500, 10.0)


def test_no_request_has_a_prefix():
    for starts in ([0, 0], [5, 5], [2, 2]):
        c = make([(200, 0)], [20, 0, 301, 64, 7], 8, 2, 1, 128, 16, seed=2)
        c["prefix_starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        out = call(c)
        check_no_device_error()
        check(out, reference(c), "bf16", 301, 10.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
def test_most_prefixes(kind):
    prefixes = [(1 + (53 * i) % 290, 1 + i % 2) for i in range(256)]
    lens = [n + (7 * i) % 20 for i, (n, k) in enumerate(prefixes) for _ in range(k)]
    c = make(prefixes, lens, 8, 2, 1, 128, 16, seed=3, pool=kind)
    out = call(c, kind)
    check_no_device_error()
    check(out, reference(c, kind), kind, max(lens), 10.0)


@pytest.mark.parametrize("kind,row", [("bf16", 256), ("e4m3", 128), ("q4", ROW)])
def test_offsets_past_32_bits(kind, row):
    """The prefix's pages and the requests' own behind byte 2^32 of the pools."""
    c = make([(300, 3)], [310, 301, 400], 8, 2, 1, 128, 16, seed=4, pool=kind)
    used = c["key_pages"].shape[0]
    P = (1 << 32) // (2 * 16 * row) + 64
    for x in ("key_pages", "value_pages"):
        big = torch.empty((P, *c[x].shape[1:]), dtype=c[x].dtype, device="cuda")
        big.view(torch.uint8).fill_(0xFF)
        big[P - used:] = c[x]
        c[x] = big
    for x in ("block_table", "prefix_table"):
        c[x][c[x] >= 0] += P - used
    out = call(c, kind)
    check_no_device_error()
    check(out, reference(c, kind), kind, 400, 10.0)


def test_append_of_more_rows_than_blocks():
    """65535 blocks take 16 rows each; the rows behind them go round again."""
    import paged_kv_attention_06_gb300 as pa
    L, H, ps = 140000, 8, 16
    x = torch.randn(1, H, L, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    k = x.to(torch.bfloat16)
    v = k.flip(-1).contiguous()
    slots = torch.randperm(L, device="cuda").to(torch.int32)[None]
    pools = [[torch.zeros((L // ps, H, ps, ROW), dtype=torch.uint8, device="cuda") for _ in "kv"] for _ in range(2)]
    pa.pa_append_kv_q4(k, v, *pools[0], slots, ps)
    for a in range(0, L, 35000):
        part = slice(a, a + 35000)
        pa.pa_append_kv_q4(k[:, :, part].contiguous(), v[:, :, part].contiguous(), *pools[1],
                           slots[:, part].contiguous(), ps)
    check_no_device_error()
    assert all(torch.equal(x, y) for x, y in zip(*pools))


def test_read_back_into_too_few_rows():
    """A context longer than the dense rows is recorded and cut."""
    import paged_kv_attention_06_gb300 as pa
    from q4_ref import dense_values, make as make_q4
    c = make_q4([300, 100], 4, 2, 1, 16, seed=6)
    kd, _ = pa.pa_gather_kv_q4(c["key_pages"], c["value_pages"], c["block_table"], c["context_lens"], 16, 130)
    assert pa.pa_get_device_error() == (pa.PA_ERR_DEVICE_BOUNDS, pa.PA_DEVERR_CONTEXT_LEN)
    j = torch.arange(130, device="cuda")
    rows = c["key_pages"][c["block_table"][0, j // 16].long(), :, j % 16].transpose(0, 1).cpu().numpy()
    assert torch.equal(kd[0].double().cpu(), torch.from_numpy(dense_values(rows)))


def test_host_threads():
    """First and later calls of every pool type from eight threads, each on a stream of its own."""
    cases = [(k, make([(400 + 100 * i, 5)], [401 + 100 * i + 9 * j for j in range(5)], 8, 2, 1, 128, 16, 40 + i, k))
             for i in range(3) for k in ("bf16", "e4m3", "q4")][:8]
    torch.cuda.synchronize()
    outs, errors = [None] * len(cases), []

    def work(i):
        try:
            kind, c = cases[i]
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                outs[i] = [call(c, kind) for _ in range(10)]
            side.synchronize()
        except Exception as e:                               # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    check_no_device_error()
    for (kind, c), got in zip(cases, outs):
        check(got[0], reference(c, kind), kind, 800, 10.0)
        assert all(torch.equal(got[0], x) for x in got)


def test_workspace_of_refused_sizes_is_zero():
    import paged_kv_attention_06_gb300 as pa
    good = dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, q_len=4, num_pages=64, max_pages=8)

    def sizes_of(**other):
        shape = pa.pa_shape(*(dict(good, **other)[f] for f, *_ in pa.pa_shape._fields_))
        return (pa.pa_decode_q4_workspace_bytes(shape), pa.pa_prefill_q4_workspace_bytes(shape, 100),
                pa.pa_attention_q4_workspace_bytes(shape, 100),
                pa.pa_decode_prefix_q4_workspace_bytes(shape, 16, 1, 100))

    assert all(sizes_of())
    for L in (4, 300):
        for bad in (dict(num_q_heads=5), dict(num_q_heads=0), dict(num_kv_heads=0), dict(num_q_heads=-4),
                    dict(q_len=0), dict(q_len=-3), dict(batch=0), dict(head_dim=64)):
            assert not any(sizes_of(**dict(dict(q_len=L), **bad))), bad
