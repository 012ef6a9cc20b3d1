"""The prefills that hand states from block to block (pa_attention's tail pieces,
pa_prefill_split), captured and replayed on other inputs: the launch's stamp is
the same in every replay, so the states that the replay before left must not be
taken for this one's."""
import pytest
import torch

from window_ref import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("setting", [4, 5])
def test_tail_pieces_in_a_replayed_graph_see_new_inputs(setting):
    import paged_kv_attention_06_gb300 as pa
    lens = [3000, 700, 2600, 300, 129]
    c = make(lens, 4, 2, 129, 128, 16, 60, poison=False)
    fresh = make(lens, 4, 2, 129, 128, 16, 61, poison=False)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["query"])

    def call(c, out, ws):
        return pa.pa_attention(**c, max_context_len=3000, out=out, workspace=ws)

    pa.pa_debug_prefill_variant(setting)
    try:
        call(c, out, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(c, out, ws)
        graph.replay()
        want = call(fresh, torch.empty_like(out), torch.zeros_like(ws))
        for k in ("query", "key_pages", "value_pages", "block_table"):
            c[k].copy_(fresh[k])
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    finally:
        pa.pa_debug_prefill_variant(0)


@pytest.mark.parametrize("lens, L", [([3000], 129), ([2600, 900], 200), ([9000], 64), ([700, 300, 2900], 130)])
def test_split_prefill_in_a_replayed_graph_sees_new_inputs(lens, L):
    import paged_kv_attention_06_gb300 as pa
    c = make(lens, 4, 2, L, 128, 16, 62, poison=False)
    fresh = make(lens, 4, 2, L, 128, 16, 63, poison=False)
    out = torch.empty_like(c["query"])
    ws, _ = pa.prefill_workspace(pa.make_shape(c["query"].shape, c["key_pages"].shape, c["block_table"].shape[1]), 16,
                                 c["query"].device)

    def call(c, out, ws):
        return pa.pa_prefill_split(**c, out=out, workspace=ws)

    call(c, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, out, ws)
    graph.replay()
    want = call(fresh, torch.empty_like(out), torch.zeros_like(ws))
    for k in ("query", "key_pages", "value_pages", "block_table"):
        c[k].copy_(fresh[k])
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
