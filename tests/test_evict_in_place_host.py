"""pa_kv_evict in place: the block table is its own destination, so both have one row
width. Argument checks through the C ABI, without a GPU."""
import pytest

from test_evict_host import GOOD, SHAPE, Shape, lib  # noqa: F401

PA_ERR_INVALID_ARG = 1


def call(f, **change):
    a = dict(GOOD, dst=GOOD["bt"], **{k: v for k, v in change.items() if k != "batch"})
    s = Shape(**dict(SHAPE, batch=change.get("batch", SHAPE["batch"])))
    return f(*[a[k] for k in ("kp", "vp", "wp", "bt", "cl", "ps", "keep", "sinks", "recent", "dst",
                              "dmp", "kept", "nl")], s, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("width", [3, 7, 9])
def test_a_table_of_another_width_is_refused(lib, fp8, width):  # noqa: F811
    f = lib.pa_kv_evict_fp8 if fp8 else lib.pa_kv_evict
    assert call(f, dmp=width) == PA_ERR_INVALID_ARG


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("change", [dict(dmp=8), dict(dmp=3, batch=1), dict(dmp=9, batch=1)])
def test_the_same_width_or_one_request_pass_the_checks(lib, fp8, change):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are no memory: only the checks before the launch are tested")
    f = lib.pa_kv_evict_fp8 if fp8 else lib.pa_kv_evict
    assert call(f, **change) != PA_ERR_INVALID_ARG
