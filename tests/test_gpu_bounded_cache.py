"""The bounded-cache calls together, as a serving loop uses them: projection rows
to the cache (norms, rotation, append), attention, and the cache held to a
bound, by a sliding window whose pages go back to the allocator, or by evicting
the slots of least accumulated weight. Everything is compared with 64-bit
arithmetic on the whole history.

Tolerances: outputs and weights as in window_ref and test_gpu_weights (the
reference reads the K/V rows that the append stored, themselves checked against
the formula in test_gpu_norm_rope). Which slots are evicted follows from the
stored weights, bit for bit.
"""
import math

import numpy as np
import pytest
import torch

from gpu_util import check_no_device_error
from window_ref import F8, SCALES

pytestmark = pytest.mark.gpu
H_Q, H_KV, D, PS = 8, 2, 128, 16
G = H_Q // H_KV


def _pa():
    import paged_kv_attention_06_gb300 as pa
    return pa


class Loop:
    """Weights of one layer, pools, allocator, and the history that the
    reference attends to: per request and KV head the stored K/V rows."""

    def __init__(self, pages, fp8, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.fp8 = g, fp8
        self.cache = _pa().KVCache(pages, PS)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in "qk")
        angle = torch.arange(4096, device="cuda", dtype=torch.float64)[:, None] * \
            (10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        shape = (pages, H_KV, PS, D)
        # pages that were never written, or hold another request's rows, are NaN
        if fp8:
            self.kp, self.vp = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv")
        else:
            self.kp, self.vp = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.wp = torch.full(shape[:3], float("nan"), device="cuda")
        self.scales = dict(k_scale=SCALES[0], v_scale=SCALES[1]) if fp8 else {}
        self.text = {}                    # tokens seen so far, by request (positions)

    def wide(self, pool, scale):
        return pool.view(F8).float().double() * scale if self.fp8 else pool.double()

    def append(self, ids, L):
        """L new tokens for every request: (queries, block table, lengths, slots)."""
        pa = _pa()
        bt, cl, sm = self.cache.plan(ids, [L] * len(ids), 64, L)
        bt, cl, sm = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (bt, cl, sm))
        qkv = (torch.randn((len(ids), L, (H_Q + 2 * H_KV) * D), generator=self.g, device="cuda")).to(torch.bfloat16)
        pos = torch.tensor([[self.text.get(i, 0) + t for t in range(L)] for i in ids], dtype=torch.int32, device="cuda")
        f = pa.pa_qk_norm_rope_append_fp8 if self.fp8 else pa.pa_qk_norm_rope_append
        q = f(qkv, self.wq, self.wk, self.cos_sin, pos, self.kp, self.vp, sm, PS, **self.scales)
        for i in ids:
            self.text[i] = self.text.get(i, 0) + L
        return q, bt, cl, sm

    def stored(self, sm):
        """The rows at slots sm [n]: K and V [H_kv, n, D] in 64 bits."""
        s = sm.long()
        return tuple(self.wide(p[s // PS, :, s % PS], sc).transpose(0, 1)
                     for p, sc in ((self.kp, SCALES[0]), (self.vp, SCALES[1])))


def attend(q, k, v, seen):
    """q [H_q, L, D], k and v [H_kv, n, D], seen [L, n]: (out, sum p |v|, score
    size, weights [H_kv, n])."""
    k, v = (x.repeat_interleave(G, 0) for x in (k, v))
    z = (q.double() @ k.transpose(1, 2)) / math.sqrt(D)
    p = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
    size = float((q.double().abs() @ k.abs().transpose(1, 2)).max() / math.sqrt(D))
    return p @ v, p @ v.abs(), size, p.view(H_KV, G, *p.shape[1:]).sum((1, 2))


def near(out, ref, mag, size, n, p_err):
    tol = ref.abs() * 2.0 ** -8 + mag * (p_err + size * 2.0 ** -15 + n * 2.0 ** -24) + n * 2.0 ** -25 * 9
    assert torch.isfinite(out).all()
    assert torch.all((out.double() - ref).abs() <= tol)


@pytest.mark.parametrize("fp8", [False, True])
def test_sliding_window_with_pages_given_back(fp8):
    pa = _pa()
    W, S = 100, 4
    # 560 tokens a request never fit at once: pages come back and change hands
    loop = Loop(pages=3 * 16, fp8=fp8, seed=1)
    ids = [5, 6, 7]
    hist = {i: [torch.zeros((H_KV, 0, D), dtype=torch.float64, device="cuda")] * 2 for i in ids}
    for i in ids:
        loop.cache.add(i)
    call = pa.pa_attention_window_fp8 if fp8 else pa.pa_attention_window
    for L in [37, 1, 3, 60, 1, 1, 20, 90, 1] + [1, 40, 2] * 8 + [1, 1]:
        q, bt, cl, sm = loop.append(ids, L)
        n = int(cl[0])
        out = call(q, loop.kp, loop.vp, bt, cl, PS, **loop.scales, window=W, sinks=S, max_context_len=n)
        check_no_device_error()
        at = n - L + torch.arange(L, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        seen = (j <= at) & ((j > at - W) | (j < S))
        for b, i in enumerate(ids):
            hist[i] = [torch.cat([old, new], 1) for old, new in zip(hist[i], loop.stored(sm[b]))]
            ref, mag, size, _ = attend(q[b], *hist[i], seen)
            near(out[b], ref, mag, size, W + S + L, 2.0 ** -8)
            loop.cache.trim_window(i, W, S)
    assert n == 560
    assert loop.cache.free_pages >= 3 * 16 - 3 * (1 + (W + PS - 1) // PS + 1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("decay", [1.0, 0.8])
def test_eviction_by_accumulated_weight(fp8, decay):
    pa = _pa()
    keep, S, R = 64, 2, 8
    loop = Loop(pages=40, fp8=fp8, seed=2)
    ids = [1, 2, 3]
    for i in ids:
        loop.cache.add(i)
    call = pa.pa_decode_weights_fp8 if fp8 else pa.pa_decode_weights
    evict = pa.pa_kv_evict_fp8 if fp8 else pa.pa_kv_evict
    hist = {i: [torch.zeros((H_KV, 0, D), dtype=torch.float64, device="cuda")] * 2 for i in ids}
    score = {i: torch.zeros((H_KV, 0), dtype=torch.float64, device="cuda") for i in ids}
    for step, L in enumerate([50, 1, 1, 20, 1, 1, 1, 30] + [1] * 6 + [3, 2, 40, 1]):
        q, bt, cl, sm = loop.append(ids, L)
        n = int(cl[0])
        d = 0.0 if step == 0 else decay
        out = call(q, loop.kp, loop.vp, loop.wp, bt, cl, PS, **loop.scales, max_context_len=n, decay=d)
        check_no_device_error()
        at = n - L + torch.arange(L, device="cuda")[:, None]
        seen = torch.arange(n, device="cuda") <= at
        page, off = torch.arange(n, device="cuda") // PS, torch.arange(n, device="cuda") % PS
        for b, i in enumerate(ids):
            hist[i] = [torch.cat([old, new], 1) for old, new in zip(hist[i], loop.stored(sm[b]))]
            ref, mag, size, w = attend(q[b], *hist[i], seen)
            near(out[b], ref, mag, size, n, 2.0 ** -8)
            old = torch.cat([score[i] * d, torch.zeros((H_KV, L), dtype=torch.float64, device="cuda")], 1)
            got = loop.wp[bt[b].long()[page], :, off].double().T
            tol = w * (size * 2.0 ** -15 + n * 2.0 ** -24 + 2.0 ** -20) + old * 2.0 ** -23 + 1e-34
            assert torch.all((got - (old + w)).abs() <= tol)
            score[i] = got               # the stored ones decide what is evicted
        if n > keep:
            kept, new_lens = evict(loop.kp, loop.vp, loop.wp, bt, cl, PS, keep, S, R)
            check_no_device_error()
            assert new_lens.tolist() == [keep] * len(ids)
            for b, i in enumerate(ids):
                loop.cache.truncate(i, keep)
                rows = []
                for h in range(H_KV):
                    order = sorted(range(S, n - R), key=lambda j: (-float(score[i][h, j]), j))[:keep - S - R]
                    want = list(range(S)) + sorted(order) + list(range(n - R, n))
                    assert kept[b, h].tolist() == want
                    rows.append(want)
                pick = torch.tensor(rows, device="cuda")
                hist[i] = [x.gather(1, pick[:, :, None].expand(-1, -1, D)) for x in hist[i]]
                score[i] = score[i].gather(1, pick)
    assert loop.text[1] > 150 and loop.cache.context_len(1) <= keep + 1


def test_a_step_captured_and_replayed():
    """One decode step of all four calls in one graph: replayed on other inputs
    it gives what the calls give one by one."""
    pa = _pa()
    g = torch.Generator(device="cuda").manual_seed(3)
    B, n0, keep = 3, 200, 128
    counts = (n0 + PS) // PS + 1

    def state(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        P = B * counts + 2
        s = dict(kp=torch.randn((P, H_KV, PS, D), generator=g, device="cuda").to(torch.bfloat16),
                 vp=torch.randn((P, H_KV, PS, D), generator=g, device="cuda").to(torch.bfloat16),
                 wp=torch.rand((P, H_KV, PS), generator=g, device="cuda"),
                 bt=torch.randperm(P, generator=g, device="cuda")[:B * counts].view(B, counts).to(torch.int32),
                 qkv=torch.randn((B, 1, (H_Q + 2 * H_KV) * D), generator=g, device="cuda").to(torch.bfloat16),
                 w=torch.rand(D, generator=g, device="cuda").to(torch.bfloat16),
                 cs=torch.randn((400, D), generator=g, device="cuda"),
                 pos=torch.randint(0, 400, (B, 1), generator=g, device="cuda").to(torch.int32),
                 cl=torch.tensor([n0, n0 - 50, n0 - 99], dtype=torch.int32, device="cuda"))
        last = s["cl"].long()[:, None] - 1
        s["sm"] = (s["bt"].gather(1, last // PS).long() * PS + last % PS).to(torch.int32)
        return s

    def run(s):
        q = pa.pa_qk_norm_rope_append(s["qkv"], s["w"], s["w"], s["cs"], s["pos"], s["kp"], s["vp"], s["sm"], PS)
        a = pa.pa_attention_window(q, s["kp"], s["vp"], s["bt"], s["cl"], PS, window=64, sinks=4, max_context_len=n0)
        b = pa.pa_decode_weights(q, s["kp"], s["vp"], s["wp"], s["bt"], s["cl"], PS, max_context_len=n0)
        kept, lens = pa.pa_kv_evict(s["kp"], s["vp"], s["wp"], s["bt"], s["cl"], PS, keep, 4, 16)
        return [q, a, b, kept, lens, s["kp"], s["vp"], s["wp"]]

    live = state(10)
    run(live)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(live)
    for seed in (11, 12):
        fresh = state(seed)
        for k, v in fresh.items():
            live[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = run(fresh)
        check_no_device_error()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("call", ["append", "window", "workspace", "evict"])
def test_memory_made_for_another_stream_is_not_in_use_on_this_one(call):
    """A tensor freed on the current stream while a copy of it is still to run
    there: the memory that a call on another stream makes is not that one."""
    pa = _pa()
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, L = 64, 64 if call == "append" else 1
    kp, vp = (torch.randn((8, H_KV, PS, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    wp = torch.rand((8, H_KV, PS), generator=gen, device="cuda")
    ids = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn((1, H_Q, L, D), generator=gen, device="cuda").to(torch.bfloat16)
    qkv = torch.randn((1, L, (H_Q + 2 * H_KV) * D), generator=gen, device="cuda").to(torch.bfloat16)
    slots = torch.arange(L, dtype=torch.int32, device="cuda")[None]
    side = torch.cuda.Stream()
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    raw = side.cuda_stream
    if call == "append":
        run = lambda: pa.pa_qk_norm_rope_append(qkv, None, None, None, None, kp, vp, slots, PS, stream=raw)
        size = q.nbytes
    elif call == "window":
        run = lambda: pa.pa_decode_window(q, kp, vp, ids, lens, PS, 32, 2, max_context_len=n, workspace=ws,
                                          stream=raw)
        size = q.nbytes
    elif call == "workspace":
        run = lambda: pa.pa_decode_weights(q, kp, vp, wp, ids, lens, PS, n, decay=0.0, out=out, stream=raw)
        shape = pa.make_shape(q.shape, kp.shape, ids.shape[1])
        size = pa.pa_decode_weights_workspace_bytes(shape, n)
    else:
        run = lambda: pa.pa_kv_evict(kp, vp, wp, ids, lens, PS, 32, 2, 8, stream=raw)
        size = H_KV * 32 * 4
    run()                                            # loads the kernels
    torch.cuda.synchronize()
    held = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                   # about 0.1 s
    copy = held.clone()
    del held
    run()
    torch.cuda.synchronize()
    check_no_device_error()
    assert torch.all(copy == 7)
