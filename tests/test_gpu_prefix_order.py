"""Decode behind shared prefixes right behind the kernels that write what it reads. The
few-row kernel of the call starts before the kernel in front of it has ended; it must see
queries, lengths, tables and rows as they were written, not as the call before left them in
a cache."""
import pytest
import torch

from gpu_util import check_no_device_error
from prefix_ref import make

pytestmark = pytest.mark.gpu

FIELDS = ("query", "key_pages", "value_pages", "block_table", "context_lens", "prefix_table", "prefix_lens",
          "prefix_starts")


def calls(kind):
    import paged_kv_attention_06_gb300 as pa
    from window_ref import SCALES
    f = {"bf16": pa.pa_decode_prefix, "e4m3": pa.pa_decode_prefix_fp8, "q4": pa.pa_decode_prefix_q4}[kind]
    return lambda c, **kw: f(**c, **(dict(k_scale=SCALES[0], v_scale=SCALES[1]) if kind == "e4m3" else {}), **kw)


def inputs(kind, seed):
    """One shape, other values, lengths, groups and places of the pages for each seed."""
    a, b = 3 + seed % 4, 9 - seed % 4
    plens = [200 + 16 * (seed % 5), 700 - 32 * (seed % 3)]
    lens = [plens[0] + 1 + (11 * i + 7 * seed) % 90 for i in range(a)]
    lens += [plens[1] + 1 + (13 * i + 5 * seed) % 150 for i in range(b)]
    c = make([(plens[0], a), (plens[1], b)], lens, 8, 2, 1, 128, 16, 100 + seed, kind)
    wide = {"key_pages": (0, 300), "value_pages": (0, 300), "block_table": (1, 60), "prefix_table": (1, 50)}
    for name, (dim, n) in wide.items():
        x = c[name]
        pad = list(x.shape)
        pad[dim] = n - pad[dim]
        fill = -1 if x.dtype == torch.int32 else 0
        c[name] = torch.cat([x, torch.full(pad, fill, dtype=x.dtype, device="cuda")], dim).contiguous()
    return c


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "q4"])
@pytest.mark.parametrize("captured", [False, True])
def test_inputs_written_just_before(kind, captured):
    call = calls(kind)
    sets = [inputs(kind, seed) for seed in range(6)]
    wants = []
    for c in sets:
        wants.append(call(c, max_context_len=900))
        torch.cuda.synchronize()
    live = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in sets[0].items()}
    source = {k: torch.stack([c[k].view(torch.uint8) if c[k].dtype == torch.bfloat16 else c[k] for c in sets])
              for k in FIELDS}
    which = torch.zeros((), dtype=torch.long, device="cuda")
    out = torch.empty_like(wants[0])

    def step():
        for k in FIELDS:
            to = live[k].view(torch.uint8) if live[k].dtype == torch.bfloat16 else live[k]
            torch.index_select(source[k], 0, which.view(1), out=to.view(1, *to.shape))
        call(live, max_context_len=900, out=out)

    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    results = []
    order = [(5 * i + i // 6) % 6 for i in range(60)]
    for i in order:
        which.fill_(i)
        graph.replay() if captured else step()
        results.append(out.clone())
    check_no_device_error()
    for i, got in zip(order, results):
        assert torch.equal(got, wants[i]), i
