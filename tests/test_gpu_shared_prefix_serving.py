"""The 4-bit pages and the decode behind shared prefixes as a server uses them together: one
prompt written once, requests that go on from it, tokens appended and attended to step by
step, a captured step, several calls on their way at once."""
import numpy as np
import pytest
import torch

from gpu_util import check_no_device_error
from prefix_ref import check, make, reference
from q4_ref import dense_values, quantise

pytestmark = pytest.mark.gpu

D, PS = 128, 16



def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


class Server:
    """Requests behind one prefix. quant: 4-bit pools, else bf16."""

    def __init__(self, prefix, own, room, H_q, H_kv, quant, seed):
        self.pa, self.quant = _pa(), quant
        self.H_q, self.H_kv, self.prefix = H_q, H_kv, prefix
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        B, n_own = len(own), [-(-(prefix + n + room) // PS) - prefix // PS for n in own]
        shared = -(-prefix // PS)
        P = shared + sum(n_own) + 1
        ids = np.random.default_rng(seed).permutation(P)
        self.ptable = torch.from_numpy(ids[:shared].astype(np.int32))[None].cuda()
        width = max(-(-(prefix + n + room) // PS) for n in own)
        table = np.full((B, width), -1, np.int32)
        at = shared
        for b, k in enumerate(n_own):
            table[b, prefix // PS:prefix // PS + k] = ids[at:at + k]
            at += k
        self.host_table = table
        self.table = torch.from_numpy(table).cuda()
        row, t = (80, torch.uint8) if quant else (D, torch.bfloat16)
        fill = 0xFF if quant else float("nan")
        self.kp, self.vp = (torch.full((P, H_kv, PS, row), fill, dtype=t, device="cuda") for _ in "kv")
        self.lens = [prefix] * B
        self.plens = torch.tensor([prefix], dtype=torch.int32, device="cuda")
        self.starts = torch.tensor([0, B], dtype=torch.int32, device="cuda")
        k, v = self.rows(1, prefix)
        slots = ids[np.arange(prefix) // PS] * PS + np.arange(prefix) % PS
        self.append(k, v, torch.from_numpy(slots.astype(np.int32))[None].cuda())
        # a partly filled last prefix page is the requests' to copy: their tables lead to
        # their own positions only, so the first own positions start in their own page
        top = max(own)
        k, v = self.rows(B, top)
        slots = torch.from_numpy(np.stack([self.slots_of(b, prefix, n, top) for b, n in enumerate(own)])).cuda()
        self.append(k, v, slots)
        self.lens = [prefix + n for n in own]

    def slots_of(self, b, first, n, width):
        j = first + np.arange(n)
        s = self.host_table[b, j // PS] * PS + j % PS
        return np.concatenate([s, np.full(width - n, -1)]).astype(np.int32)

    def rows(self, B, n):
        return (torch.randn(B, self.H_kv, n, D, generator=self.g, device="cuda").to(torch.bfloat16) for _ in "kv")

    def append(self, k, v, slots):
        f = self.pa.pa_append_kv_q4 if self.quant else self.pa.pa_append_kv
        f(k, v, self.kp, self.vp, slots, PS)

    def case(self, q, lens):
        return dict(query=q, key_pages=self.kp, value_pages=self.vp, block_table=self.table, context_lens=lens,
                    page_size=PS, prefix_table=self.ptable, prefix_lens=self.plens, prefix_starts=self.starts)

    def decode(self, q, lens, **kw):
        f = self.pa.pa_decode_prefix_q4 if self.quant else self.pa.pa_decode_prefix
        return f(**self.case(q, lens), **kw)

    def query(self, L):
        q = torch.randn(len(self.lens), self.H_q, L, D, generator=self.g, device="cuda")
        return (q * 1.3).to(torch.bfloat16)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("prefix,L", [(640, 1), (331, 1), (331, 3)])
def test_steps_of_a_server(prefix, L, quant):
    """Each step appends L tokens a request, decodes behind the prefix, and says what the
    call over whole tables says."""
    kind = "q4" if quant else "bf16"
    s = Server(prefix, [1, 40, 17, 300, 5, 64], 4 * L, 8, 2, quant, seed=prefix + L)
    B = len(s.lens)
    whole = s.host_table.copy()                # tables with the prefix's whole pages in place
    whole[:, :prefix // PS] = s.ptable[0, :prefix // PS].cpu().numpy()
    for step in range(4):
        k, v = s.rows(B, L)
        slots = np.stack([s.slots_of(b, n, L, L) for b, n in enumerate(s.lens)])
        s.append(k, v, torch.from_numpy(slots).cuda())
        s.lens = [n + L for n in s.lens]
        lens = torch.tensor(s.lens, dtype=torch.int32, device="cuda")
        q = s.query(L)
        out = s.decode(q, lens, max_context_len=max(s.lens))
        check_no_device_error()
        ref = reference(s.case(q, lens), kind)
        check(out, ref, kind, max(s.lens), 10.0)
        if prefix % PS == 0:
            f = s.pa.pa_attention_q4 if quant else s.pa.pa_attention
            same = f(q, s.kp, s.vp, torch.from_numpy(whole).cuda(), lens, PS,
                     **(dict(max_context_len=max(s.lens)) if quant else {}))
            check_no_device_error()
            for b, (r, mag, size) in enumerate(ref):       # both within their bounds of the same
                tol = 2 * (r.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + size * 2.0 ** -15 + 2.0 ** -10))
                assert ((out[b].double() - same[b].double()).abs() <= tol).all()


def test_read_back_of_what_a_server_wrote():
    s = Server(400, [16, 90, 33], 0, 8, 2, True, seed=5)
    rng = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn(1, 2, 400, D, generator=rng, device="cuda").to(torch.bfloat16)   # the prefix's keys
    got_k, got_v = s.pa.pa_gather_kv_q4(s.kp, s.vp, s.ptable, s.plens, PS, 400)
    check_no_device_error()
    want = torch.from_numpy(dense_values(quantise(k.double().cpu().numpy()))).to(torch.bfloat16)
    assert torch.equal(got_k.cpu(), want)
    assert torch.isfinite(got_v).all()


@pytest.mark.parametrize("quant", [False, True])
def test_a_captured_step(quant):
    """Append and decode in one graph, replayed with other tokens, slots, lengths."""
    def fresh():
        return Server(500, [3, 100, 31, 200], 8, 8, 2, quant, seed=9)

    a, b = fresh(), fresh()                    # the same twice: one eager, one replayed
    B = len(a.lens)
    k, v = (torch.zeros(B, 2, 1, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q = torch.zeros(B, 8, 1, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    lens = torch.tensor(b.lens, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    b.append(k, v, slots)                      # (nothing: every slot is -1)
    b.decode(q, lens, out=out, max_context_len=720)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.append(k, v, slots)
        b.decode(q, lens, out=out, max_context_len=720)
    for step in range(5):
        nk, nv = a.rows(B, 1)
        nq = a.query(1)
        at = torch.from_numpy(np.stack([a.slots_of(i, n, 1, 1) for i, n in enumerate(a.lens)])).cuda()
        a.append(nk, nv, at)
        a.lens = [n + 1 for n in a.lens]
        now = torch.tensor(a.lens, dtype=torch.int32, device="cuda")
        want = a.decode(nq, now, max_context_len=720)
        for x, y in ((k, nk), (v, nv), (q, nq), (slots, at), (lens, now)):
            x.copy_(y)
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(out, want), step
    assert torch.equal(a.kp.view(torch.uint8), b.kp.view(torch.uint8))
    check_no_device_error()


def test_graphs_that_share_a_workspace():
    """Calls of different shapes, replayed in turn over one workspace."""
    pa = _pa()
    cases = [make([(900, 20)], [901 + 7 * i for i in range(20)], 8, 2, 1, D, PS, 21, "q4"),
             make([(300, 3), (50, 2)], [301, 400, 310, 51, 90], 4, 1, 2, D, PS, 22, "q4")]
    need = max(pa.pa_decode_prefix_q4_workspace_bytes(
        pa.make_shape(c["query"].shape, c["key_pages"].shape, c["block_table"].shape[1], q4=True), PS,
        len(c["prefix_lens"]), PS * c["prefix_table"].shape[1]) for c in cases)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    wants = [pa.pa_decode_prefix_q4(**c) for c in cases]
    outs = [torch.empty_like(w) for w in wants]
    graphs = []
    for c, out in zip(cases, outs):
        pa.pa_decode_prefix_q4(**c, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.pa_decode_prefix_q4(**c, out=out, workspace=ws)
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1, 0, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], wants[i])
    check_no_device_error()


def test_calls_on_two_streams_at_once():
    pa = _pa()
    cases = [make([(2000, 24)], [2001 + 11 * i for i in range(24)], 8, 2, 1, D, PS, 31, k) for k in ("q4", "bf16")]
    calls = [pa.pa_decode_prefix_q4, pa.pa_decode_prefix]
    wants = [f(**c) for f, c in zip(calls, cases)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for f, c, s in zip(calls, cases, streams):
            with torch.cuda.stream(s):
                outs.append(f(**c))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, wants[i % 2])
    check_no_device_error()


def test_a_prompt_behind_a_quantised_context():
    """A chunk of a prompt is appended and attended to (prefill), then single tokens behind
    it (decode) see the same cache."""
    pa = _pa()
    s = Server(256, [16, 16], 200, 8, 2, True, seed=41)
    B, L = 2, 150
    whole = s.host_table.copy()
    whole[:, :256 // PS] = s.ptable[0].cpu().numpy()
    table = torch.from_numpy(whole).cuda()
    k, v = s.rows(B, L)
    s.append(k, v, torch.from_numpy(np.stack([s.slots_of(b, n, L, L) for b, n in enumerate(s.lens)])).cuda())
    s.lens = [n + L for n in s.lens]
    lens = torch.tensor(s.lens, dtype=torch.int32, device="cuda")
    q = s.query(L)
    out = pa.pa_attention_q4(q, s.kp, s.vp, table, lens, PS, max_context_len=max(s.lens))
    last = pa.pa_attention_q4(q[:, :, -1:].contiguous(), s.kp, s.vp, table, lens, PS, max_context_len=max(s.lens))
    shared = s.decode(q[:, :, -1:].contiguous(), lens, max_context_len=max(s.lens))
    check_no_device_error()
    c = s.case(q[:, :, -1:].contiguous(), lens)
    ref = reference(c, "q4")
    check(shared, ref, "q4", max(s.lens), 10.0)
    for b, (r, mag, size) in enumerate(ref):
        # the prefill's keys are rounded to bf16 (2^-9 of the scores' terms, on both sides)
        tol = 2 * (r.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + size * 2.0 ** -7))
        for got in (out[b, :, -1:], last[b]):
            assert ((got.double() - r).abs() <= tol).all()
