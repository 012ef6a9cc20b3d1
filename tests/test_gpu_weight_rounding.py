"""The softmax's weights over codes, and the values of 4-bit rows, are held in f16, not in
bf16. Random numbers do not tell the two apart: the errors average out below the output's
own rounding. Here they add up. Weights: of every 16 keys two have weight 1 and the value 0,
seven a weight that bf16 rounds down and the value 1, seven a weight that it rounds up and the
value -1. Values: all weights 1, half the values one that bf16 rounds up, half the negative
of one that it rounds down."""
import math

import pytest
import torch

from gpu_util import check_no_device_error
from prefix_ref import make as make_prefix, reference as prefix_reference
from q4_ref import make as make_q4, reference as q4_reference
from window_ref import F8, SCALES

DOWN, UP = 0.5 + 3 * 2.0 ** -11, 0.5 + 5 * 2.0 ** -11      # f16 has both; bf16 has 1/2 and 1/2 + 2^-8
WEIGHTS = [1.0] + [DOWN, UP] * 7 + [1.0]
VALUES = [0.0] + [1.0, -1.0] * 7 + [0.0]
HIGH, LOW = 1 + 3 * 2.0 ** -9, 1 + 2.0 ** -9               # bf16 has 1 and 1 + 2^-7
QUERY = [2.0 ** (3 - 4 * d) for d in range(4)]             # at elements 0, 32, 64 and 96; zeros elsewhere


def digits(weight, k_scale):
    """Key elements 0, 32, 64, 96 in e4m3, so that the score is ln(weight) to about 2^-16."""
    rest, out = math.log(weight) * math.sqrt(128) / k_scale, []
    for q in QUERY:
        v = float(torch.tensor(rest / q).to(F8).float())
        out.append(v)
        rest -= v * q
    assert abs(rest) * k_scale / math.sqrt(128) < 2.0 ** -16
    return out


def fill(c, kind, weights=WEIGHTS, values=VALUES):
    """Every page 16 keys of these weights and values, every query row QUERY."""
    k_scale = SCALES[0] if kind == "e4m3" else 1.0
    keys, values = torch.zeros(16, 128), torch.tensor(values)[:, None].expand(16, 128)
    for i, w in enumerate(weights):
        keys[i, ::32] = torch.tensor(digits(w, k_scale))
    for name, x in (("key_pages", keys), ("value_pages", values)):
        if kind == "e4m3":
            rows = x.to(F8).view(torch.uint8)
        else:                                              # steps of 0: a group is its least value
            least = x[:, ::32]
            parts = torch.stack([torch.zeros_like(least), least], -1).flatten(1).half()
            rows = torch.zeros(16, 80, dtype=torch.uint8)
            rows[:, 64:] = parts.contiguous().view(torch.uint8)
        c[name] = rows.to(c[name].device).expand(*c[name].shape).contiguous()
    q = torch.zeros(128)
    q[::32] = torch.tensor(QUERY)
    c["query"] = q.to(torch.bfloat16).to(c["query"].device).expand(*c["query"].shape).contiguous()
    return c


def check(out, ref, n_max, v_scale=1.0):
    """Output rounding 2^-8 of the value; a weight's 2^-11 (f16, half a step), so 2^-11 of
    sum p |v|, and 2^-25 a key where it is subnormal; scores and sums in fp32 as prefix_ref.check has
    them."""
    for b, (r, mag, size, *_) in enumerate(ref):
        tol = r.abs() * 2.0 ** -8 + mag * (2.0 ** -11 + size * 2.0 ** -15 + n_max * 2.0 ** -24 + 2.0 ** -20)
        tol = tol + n_max * 2.0 ** -25 * v_scale + 1e-30
        err = (out[b].double() - r).abs()
        assert torch.all(err <= tol), (b, float((err / tol).max()))


def test_the_bound_tells_the_two_apart():
    """On the CPU: these weights as f16 lie within it, as bf16 several times beyond."""
    p = torch.tensor(WEIGHTS * 40, dtype=torch.float64)
    v = torch.tensor(VALUES * 40, dtype=torch.float64)
    r, mag = (p @ v) / p.sum(), (p @ v.abs()) / p.sum()
    ref = [(r[None], mag[None], 1.0)]
    check([((p.half().double() @ v) / p.sum())[None]], ref, len(p))
    bf16 = ((p.to(torch.bfloat16).double() @ v) / p.sum())[None]
    with pytest.raises(AssertionError):
        check([bf16], ref, len(p))
    assert float((bf16 - r).abs()) > 4 * float(mag) * 2.0 ** -11
    v = torch.tensor([HIGH, -LOW] * 300, dtype=torch.float64)
    r, mag = v.mean(), v.abs().mean()
    check([v.half().double().mean()[None]], [(r[None], mag[None], 1.0)], len(v))
    with pytest.raises(AssertionError):
        check([v.to(torch.bfloat16).double().mean()[None]], [(r[None], mag[None], 1.0)], len(v))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,what", [("e4m3", "weights"), ("q4", "weights"), ("q4", "values")])
@pytest.mark.parametrize("prefix,requests,L", [(160, 3, 1), (2048, 20, 1), (2048, 40, 1), (640, 4, 4)])
def test_behind_a_prefix(prefix, requests, L, kind, what):
    import paged_kv_attention_06_gb300 as pa
    lens = [prefix + 16 * (1 + i % 5) for i in range(requests)] + [320]
    c = make_prefix([(prefix, requests)], lens, 8, 2, L, 128, 16, 1, kind, poison=False)
    c = fill(c, kind) if what == "weights" else fill(c, kind, [1.0] * 16, [HIGH, -LOW] * 8)
    if kind == "e4m3":
        out = pa.pa_decode_prefix_fp8(**c, k_scale=SCALES[0], v_scale=SCALES[1])
    else:
        out = pa.pa_decode_prefix_q4(**c)
    check_no_device_error()
    check(out, prefix_reference(c, kind), max(lens), SCALES[1] if kind == "e4m3" else 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["weights", "values"])
@pytest.mark.parametrize("L", [1, 4, 40, 300, 700])
def test_over_4_bit_pages(L, what):
    """Decode, split prefill and (700 rows, 6 requests of 32 heads) the kernel of pairs."""
    import paged_kv_attention_06_gb300 as pa
    lens, H_q, H_kv = ([L + 16 * i for i in range(6)], 32, 8) if L == 700 else ([L + 200, L + 8, L], 8, 2)
    c = make_q4(lens, H_q, H_kv, L, 16, 1, poison=False)
    c = fill(c, "q4") if what == "weights" else fill(c, "q4", [1.0] * 16, [HIGH, -LOW] * 8)
    out = pa.pa_attention_q4(**c, max_context_len=max(lens))
    check_no_device_error()
    check(out, q4_reference(c, copied=L > 8), max(lens))
