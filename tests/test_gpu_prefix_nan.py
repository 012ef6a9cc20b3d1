"""NaN scores behind shared prefixes: a row that sees one is NaN, as pa_decode's is, however
the keys are cut into pieces; every other row is as it would be without."""
import pytest
import torch

from gpu_util import check_no_device_error
from prefix_ref import check, make, reference

pytestmark = pytest.mark.gpu

NAN = float("nan")


def call(c, kind="bf16"):
    import paged_kv_attention_06_gb300 as pa
    from window_ref import SCALES
    f = {"bf16": pa.pa_decode_prefix, "e4m3": pa.pa_decode_prefix_fp8, "q4": pa.pa_decode_prefix_q4}[kind]
    return f(**c, **(dict(k_scale=SCALES[0], v_scale=SCALES[1]) if kind == "e4m3" else {}))


def check_but(out, ref, nan, kind, n_max):
    """nan [B, H_q, L]: the rows that are NaN. The others within prefix_ref's bounds."""
    assert out[nan].isnan().all()
    rest = out.clone()
    for b, (r, _, _) in enumerate(ref):
        rest[b][nan[b]] = r[nan[b]].to(rest.dtype)
    check(rest, ref, kind, n_max, 10.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("plen", [1, 130, 5000])
def test_a_query_of_nan(plen, kind):
    lens = [plen + x for x in (1, 0, 30, 200, 7)]
    c = make([(plen, 4)], lens, 8, 2, 2, 128, 16, seed=plen, pool=kind)
    ref = reference(c, kind)
    nan = torch.zeros(5, 8, 2, dtype=torch.bool, device="cuda")
    nan[0, 3, 1] = nan[3, 0, 0] = nan[4, 7, 1] = True
    if plen > 1:
        nan[1, 5, 0] = True
    c["query"][nan] = NAN
    out = call(c, kind)
    check_no_device_error()
    check_but(out, ref, nan, kind, max(lens))


@pytest.mark.parametrize("many", [1, 20])
def test_keys_of_nan(many):
    """The only key of a prefix, every key of one piece, the only key of a request's own."""
    lens = [1 + i % 3 + 1 for i in range(many)] + [300 + 1 + i % 5 for i in range(many)] + [9, 40]
    c = make([(1, many), (300, many)], lens, 8, 2, 1, 128, 16, seed=many)
    ref = reference(c)
    nan = torch.zeros(len(lens), 8, 1, dtype=torch.bool, device="cuda")
    c["key_pages"][c["prefix_table"][0, 0].item(), 1, 0] = NAN          # KV head 1: query heads 4 .. 7
    nan[:many, 4:] = True
    b = many                                                            # 300 + 1 positions: one own key
    c["key_pages"][c["block_table"][b, 300 // 16].item(), 0, 300 % 16] = NAN
    nan[b, :4] = True
    out = call(c)
    check_no_device_error()
    check_but(out, ref, nan, "bf16", max(lens))


def test_keys_behind_a_shorter_request():
    """A key of NaN in the prefix makes NaN of the rows that see it; requests, and rows of a
    chunk, that end before it are as they would be without."""
    lens = [260, 251, 250, 249, 100, 1, 0, 400]
    c = make([(260, 8)], lens, 8, 2, 2, 128, 16, seed=4)
    ref = reference(c)
    c["key_pages"][c["prefix_table"][0, 250 // 16].item(), :, 250 % 16] = NAN
    nan = torch.zeros(8, 8, 2, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for i in range(2):
            nan[b, :, i] = n - 2 + i >= 250
    out = call(c)
    check_no_device_error()
    check_but(out, ref, nan, "bf16", max(lens))
