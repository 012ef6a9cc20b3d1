"""Cases, plain forms and calls of the cache-writing and bounded-cache operators.

Four kinds of case, each one pass of a serving step's work on one layer:

  append   norms of queries and keys for each head, the position rotation, and the scatter of k and v into the pages
  window   attention with a sliding window and a few first tokens that stay visible, over paged K/V
  weights  attention over paged K/V that also accumulates the attention weight of every cached slot
  evict    eviction by accumulated weight: choose the slots to keep, move their rows to the front

`own` chooses between the plain form (torch operations in 32 bits) and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # one new token of one request (the latency of a decode step's first kernel), 7 query heads per KV head
        dict(name="append_1_token", kind="append", B=1, L=1, Hq=28, Hkv=4, D=128, ps=16, R=128, inter=False, norm=True, fp8=False, pos=4096),
        # a decode batch over e4m3 pools with large pages
        dict(name="append_b64_e4m3", kind="append", B=64, L=1, Hq=32, Hkv=8, D=128, ps=128, R=128, inter=False, norm=True, fp8=True, pos=32768),
        # prefill chunks of an odd length at far positions
        dict(name="append_chunk_4x2047", kind="append", B=4, L=2047, Hq=32, Hkv=8, D=128, ps=16, R=128, inter=False, norm=True, fp8=False, pos=100000),
        # one request, a short window: the latency of a single decode
        dict(name="window_decode_b1", kind="window", B=1, L=1, Hq=28, Hkv=4, D=128, ps=16, W=512, S=4, lo=5001, hi=5001, fp8=False),
        # a ragged decode batch, some contexts shorter than the window
        dict(name="window_decode_b32_gqa7", kind="window", B=32, L=1, Hq=28, Hkv=4, D=128, ps=16, W=1024, S=4, lo=128, hi=16384, fp8=False),
        # a large decode batch over e4m3 pools with large pages
        dict(name="window_decode_b64_e4m3", kind="window", B=64, L=1, Hq=32, Hkv=8, D=128, ps=128, W=2048, S=16, lo=1000, hi=32768, fp8=True),
        # prefill chunks after ragged prefixes
        dict(name="window_prefill_4x512", kind="window", B=4, L=512, Hq=32, Hkv=8, D=128, ps=16, W=1024, S=4, lo=512, hi=2560, fp8=False),
        # a long prompt in one call, of an odd length
        dict(name="window_prefill_8191", kind="window", B=1, L=8191, Hq=32, Hkv=8, D=128, ps=16, W=2048, S=4, lo=8191, hi=8191, fp8=False),
        # a ragged decode batch that keeps the weight of every slot
        dict(name="weights_b32_gqa7", kind="weights", B=32, L=1, Hq=28, Hkv=4, D=128, ps=16, lo=128, hi=4096, decay=1.0, fp8=False),
        # long contexts over e4m3 pools, older weights fading
        dict(name="weights_long_b8_e4m3", kind="weights", B=8, L=1, Hq=32, Hkv=8, D=128, ps=16, lo=16384, hi=32768, decay=0.9, fp8=True),
        # one request just over its budget
        dict(name="evict_b1", kind="evict", B=1, Hkv=4, D=128, ps=16, lo=1280, hi=1280, keep=1024, S=4, recent=128, fp8=False),
        # long contexts cut to a quarter to a half
        dict(name="evict_long_b8", kind="evict", B=8, Hkv=8, D=128, ps=16, lo=16384, hi=32768, keep=8192, S=4, recent=512, fp8=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "window", "window", "weights", "evict"])
    fp8 = rng.random() < 0.3
    D = 128 if fp8 else rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    ps = rng.choice([4, 16, 16, 32, 64, 128, 256])
    if kind == "append":
        B = _log(rng, 1, 64)
        L = rng.choice([1, _log(rng, 1, max(1, 8000 // B))])
        return dict(kind=kind, B=B, L=L, Hq=min(Hq, 32 // Hkv * Hkv), Hkv=Hkv, D=D, ps=ps, R=rng.choice([D, D, D // 2, D // 4]), inter=rng.random() < 0.4,
                    norm=rng.random() < 0.7, fp8=fp8, pos=_log(rng, 1000, 120000))
    if kind == "window":
        Hq = min(Hq, 32 // Hkv * Hkv)
        S = rng.choice([0, 1, 4, 4, 64, 130])
        if rng.random() < 0.6:
            B, L = _log(rng, 1, 64), rng.choice([1, 1, 2, 5])
            W = _log(rng, 32, min(8192, 900000 // (B * Hkv)))
        else:
            B = _log(rng, 1, 4)
            L = _log(rng, 33, 6000 // B)
            W = _log(rng, 32, 2048)
        lo = L + _log(rng, 1, 8000)
        return dict(kind=kind, B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, ps=ps, W=W, S=S, lo=lo, hi=lo + _log(rng, 1, 8000), fp8=fp8)
    lo = _log(rng, 64, 16000)
    if kind == "weights":
        hi = lo + _log(rng, 1, 16000)
        B = _log(rng, 1, max(1, min(64, 1500000 // (Hkv * hi))))
        L = rng.choice([1, 1, 1, 2, 16, 32]) if B * Hq * hi < 500000 else 1
        return dict(kind=kind, B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, ps=ps, lo=lo, hi=hi, decay=rng.choice([1.0, 1.0, 0.9, 0.0]), fp8=fp8)
    hi = lo + _log(rng, 1, 16000)
    B = _log(rng, 1, max(1, min(64, 1500000 // (Hkv * hi))))
    keep = max(8, int(lo * rng.uniform(0.2, 1.0)))
    S = rng.choice([0, 4, min(64, keep // 4)])
    return dict(kind=kind, B=B, Hkv=Hkv, D=D, ps=ps, lo=lo, hi=hi, keep=keep, S=S, recent=rng.choice([0, 1, keep // 8, keep // 2]), fp8=fp8)


def _lengths(c):
    """Context lengths of a case: spread over [lo, hi], evenly over their logarithm."""
    lo, hi, B = c["lo"], c["hi"], c["B"]
    if B == 1:
        return [hi]
    return [min(hi, max(lo, int(round(lo * (hi / lo) ** (i / (B - 1)))))) for i in range(B)]


def _visible(c, n):
    """Positions of one request that some row of a window case sees: [0, a) and [b, n)."""
    b = max(0, n - c["L"] - c["W"] + 1)
    return min(c["S"], b), b


def work(c):
    es = 1 if c["fp8"] else 2
    if c["kind"] == "append":
        rows, heads = c["B"] * c["L"], c["Hq"] + 2 * c["Hkv"]
        return {"bytes": rows * (heads * c["D"] * 2 + c["Hq"] * c["D"] * 2 + 2 * c["Hkv"] * c["D"] * es + c["R"] * 4 + 8),
                "flops": rows * (c["Hq"] + c["Hkv"]) * (c["D"] * 4 + c["R"] * 3)}
    if c["kind"] == "evict":
        b = sum(4 * n + 4 * c["keep"] + c["keep"] * 2 * (2 * c["D"] * es + 4) for n in _lengths(c)) * c["Hkv"]
        return {"bytes": b, "flops": sum(n * c["Hkv"] for n in _lengths(c))}
    qo = c["B"] * c["L"] * c["Hq"] * c["D"] * 4
    if c["kind"] == "weights":
        keys = sum(_lengths(c))
        pairs = sum(sum(n - c["L"] + i + 1 for i in range(c["L"])) for n in _lengths(c))
        return {"bytes": qo + keys * c["Hkv"] * (2 * c["D"] * es + 4 + (4 if c["decay"] else 0)), "flops": 4 * pairs * c["Hq"] * c["D"]}
    keys = pairs = 0
    for n in _lengths(c):
        a, b = _visible(c, n)
        keys += a + n - b
        for i in range(c["L"]):
            p = n - c["L"] + i
            first = max(0, p - c["W"] + 1)
            pairs += min(c["S"], first) + p + 1 - first
    return {"bytes": qo + keys * c["Hkv"] * 2 * c["D"] * es, "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---- inputs ---------------------------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(torch.bfloat16)


def _pool(g, shape, fp8):
    x = _normal(g, shape)
    return (x.float() / 0.02).clamp(-448, 448).to(F8).view(torch.uint8) if fp8 else x


def _pages(g, counts, spare=3):
    """One row of distinct physical pages for each request, -1 behind them, and the number of pages in the pool."""
    total = sum(counts) + spare
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    width = max(counts)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, k in enumerate(counts):
        table[i, :k] = perm[at : at + k]
        at += k
    return table, total


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    D, ps, Hkv, B = c["D"], c["ps"], c["Hkv"], c["B"]
    if c["kind"] == "append":
        L, R = c["L"], c["R"]
        s["qkv"] = _normal(g, (B, L, (c["Hq"] + 2 * Hkv) * D), 1.5)
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if c["norm"] else None for _ in range(2))
        angle = torch.arange(c["pos"] + L, device=DEV, dtype=torch.float64)[:, None] * (10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        first = torch.randint(0, c["pos"], (B, 1), generator=g, device=DEV)
        s["positions"] = (first + torch.arange(L, device=DEV)).to(torch.int32)
        table, P = _pages(g, [(L + ps - 1) // ps + 1] * B)
        t = torch.randint(0, ps, (B, 1), generator=g, device=DEV) + torch.arange(L, device=DEV)
        s["slots"] = (table.gather(1, t // ps) * ps + t % ps).to(torch.int32)
        s["kp"], s["vp"] = (_pool(g, (P, Hkv, ps, D), c["fp8"]) for _ in range(2))
        s["query"] = torch.empty((B, c["Hq"], L, D), dtype=torch.bfloat16, device=DEV)
        return s
    lens = _lengths(c)
    lens = [lens[i] for i in torch.randperm(B, generator=g, device=DEV).tolist()]
    counts = [(n + ps - 1) // ps for n in lens]
    if c["kind"] == "evict":
        dst = (c["keep"] + ps - 1) // ps
        table, P = _pages(g, [k + dst for k in counts])
        s["dst"] = torch.stack([table[i, k : k + dst] for i, k in enumerate(counts)]).contiguous()
        for i, k in enumerate(counts):
            table[i, k:] = -1
    elif c["kind"] == "window":
        # a page that no row sees is not held by the request: its table entry is -1
        live = []
        for n, k in zip(lens, counts):
            a, b = _visible(c, n)
            live.append([j for j in range(k) if j * ps < a or (j + 1) * ps > b])
        rows, P = _pages(g, [len(x) for x in live])
        table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=DEV)
        for i, x in enumerate(live):
            table[i, torch.tensor(x, device=DEV)] = rows[i, : len(x)]
    else:
        table, P = _pages(g, counts)
    s["bt"] = table.contiguous()
    s["cl"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["max"] = max(lens)
    s["kp"], s["vp"] = (_pool(g, (P, Hkv, ps, D), c["fp8"]) for _ in range(2))
    if c["kind"] != "window":
        # accumulated weights: a few large, most small, some nothing at all
        u = torch.rand((P, Hkv, ps), generator=g, device=DEV)
        s["wp"] = torch.where(u < 0.02, torch.zeros_like(u), u**12 * 4)
    if c["kind"] == "evict":
        s["kept"] = torch.empty((B, Hkv, c["keep"]), dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=DEV)
    else:
        s["q"] = _normal(g, (B, c["Hq"], c["L"], D), 1.5)
        s["out"] = torch.empty_like(s["q"])
    if own:
        s["ws"] = _workspace(s)
    return s


def _workspace(s):
    import paged_kv_attention_06_gb300 as pa

    c = s["c"]
    if c["kind"] == "evict":
        return None
    shape = pa.make_shape(s["q"].shape, s["kp"].shape, s["bt"].shape[1])
    if c["kind"] == "weights":
        need = pa.pa_decode_weights_workspace_bytes(shape, s["max"])
    elif c["fp8"]:
        need = pa.pa_attention_window_fp8_workspace_bytes(shape, c["ps"], s["max"], c["W"], c["S"])
    else:
        need = pa.pa_attention_window_workspace_bytes(shape, c["ps"], s["max"], c["W"], c["S"])
    return torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)


# ---- one pass -------------------------------------------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _view(p):
    return p.view(F8) if p.dtype == torch.uint8 else p


def _own(s):
    import paged_kv_attention_06_gb300 as pa

    c = s["c"]
    scales = (0.02, 0.02) if c["fp8"] else ()
    if c["kind"] == "append":
        f = pa.pa_qk_norm_rope_append_fp8 if c["fp8"] else pa.pa_qk_norm_rope_append
        q = f(s["qkv"], s["wq"], s["wk"], s["cos_sin"], s["positions"], s["kp"], s["vp"], s["slots"], c["ps"], *scales, eps=EPS, interleaved=c["inter"], query=s["query"])
        return q, _view(s["kp"]), _view(s["vp"])
    if c["kind"] == "window":
        f = pa.pa_attention_window_fp8 if c["fp8"] else pa.pa_attention_window
        return f(s["q"], s["kp"], s["vp"], s["bt"], s["cl"], c["ps"], *scales, window=c["W"], sinks=c["S"], out=s["out"], max_context_len=s["max"], workspace=s["ws"])
    if c["kind"] == "weights":
        f = pa.pa_decode_weights_fp8 if c["fp8"] else pa.pa_decode_weights
        out = f(s["q"], s["kp"], s["vp"], s["wp"], s["bt"], s["cl"], c["ps"], *scales, max_context_len=s["max"], decay=c["decay"], out=s["out"], workspace=s["ws"])
        return out, s["wp"]
    f = pa.pa_kv_evict_fp8 if c["fp8"] else pa.pa_kv_evict
    kept, new_lens = f(s["kp"], s["vp"], s["wp"], s["bt"], s["cl"], c["ps"], keep=c["keep"], sinks=c["S"], recent=c["recent"], dst_block_table=s["dst"], kept=s["kept"], new_lens=s["new_lens"])
    return kept, new_lens, _view(s["kp"]), _view(s["vp"]), s["wp"]


def _plain(s):
    return {"append": _plain_append, "window": _plain_window, "weights": _plain_weights, "evict": _plain_evict}[s["c"]["kind"]](s)


def _store(pool, page, off, rows, scale):
    """rows [n, Hkv, D] in 32 bits into slots (page, off) of the pool."""
    if pool.dtype == torch.uint8:
        pool[page, :, off] = (rows / scale).clamp(-448, 448).to(F8).view(torch.uint8)
    else:
        pool[page, :, off] = rows.to(pool.dtype)


def _rotate(x, cos, sin, inter):
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., : R // 2], x[..., R // 2 : R])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_append(s):
    c = s["c"]
    B, L, Hq, Hkv, D, ps = (c[k] for k in ("B", "L", "Hq", "Hkv", "D", "ps"))
    x = s["qkv"].view(B, L, Hq + 2 * Hkv, D).float()
    q, k, v = x[:, :, :Hq], x[:, :, Hq : Hq + Hkv], x[:, :, Hq + Hkv :]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["wq"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["wk"].float()
    cs = s["cos_sin"][s["positions"].long()][:, :, None]
    cos, sin = cs[..., : c["R"] // 2], cs[..., c["R"] // 2 :]
    q, k = _rotate(q, cos, sin, c["inter"]), _rotate(k, cos, sin, c["inter"])
    slot = s["slots"].view(-1).long()
    _store(s["kp"], slot // ps, slot % ps, k.reshape(B * L, Hkv, D), 0.02)
    _store(s["vp"], slot // ps, slot % ps, v.reshape(B * L, Hkv, D), 0.02)
    s["query"].copy_(q.transpose(1, 2))
    return s["query"], _view(s["kp"]), _view(s["vp"])


def _rows(pool, bt, pos, ps, fp8):
    """Pool rows at positions pos [B, n] (clamped into the table where a mask hides them): [B, Hkv, n, D] in 32 bits."""
    phys = bt.gather(1, pos // ps).long().clamp_min(0)
    x = pool[phys, :, pos % ps]
    return (x.view(F8).float() * 0.02 if fp8 else x.float()).transpose(1, 2)


def _softmax_rows(s, k, seen):
    """Attention weights [B, Hkv, G, L, n] in 32 bits of the rows in s["q"] over the keys k [B, Hkv, n, D], seen [B, L, n]."""
    c = s["c"]
    q = s["q"].float().view(c["B"], c["Hkv"], -1, c["D"])
    z = (q @ k.transpose(-1, -2)) * c["D"] ** -0.5
    z = z.view(c["B"], c["Hkv"], -1, c["L"], k.shape[2]).masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp_min(-1e30))
    del z
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _times_v(s, p, v):
    c = s["c"]
    s["out"].copy_((p.view(c["B"], c["Hkv"], -1, v.shape[2]) @ v).view(s["out"].shape))
    return s["out"]


def _plain_window(s):
    c = s["c"]
    n, L, W, S = s["cl"].long()[:, None], c["L"], c["W"], c["S"]
    first = n - L - W + 1
    win = first + torch.arange(min(W + L - 1, s["max"] + W), device=DEV)
    sink = torch.arange(S, device=DEV).expand(c["B"], S)
    pos = torch.cat([sink, win], 1)
    there = torch.cat([sink < n, (win >= S) & (win < n)], 1)
    pos = torch.where(there, pos, n - 1)
    row = n - L + torch.arange(L, device=DEV)
    seen = there[:, None] & (pos[:, None] <= row[:, :, None]) & ((pos[:, None] > row[:, :, None] - W) | (pos[:, None] < S))
    p = _softmax_rows(s, _rows(s["kp"], s["bt"], pos, c["ps"], c["fp8"]), seen)
    return _times_v(s, p, _rows(s["vp"], s["bt"], pos, c["ps"], c["fp8"]))


def _plain_weights(s):
    c = s["c"]
    n, L, ps = s["cl"].long()[:, None], c["L"], c["ps"]
    pos = torch.arange(s["max"], device=DEV).expand(c["B"], -1)
    row = n - L + torch.arange(L, device=DEV)
    seen = pos[:, None] <= row[:, :, None]
    p = _softmax_rows(s, _rows(s["kp"], s["bt"], pos, ps, c["fp8"]), seen)
    out = _times_v(s, p, _rows(s["vp"], s["bt"], pos, ps, c["fp8"]))
    w = p.sum((2, 3))
    # a place behind the pool takes what lies behind a context
    pool = torch.cat([s["wp"].view(-1), s["wp"].new_zeros(1)])
    phys = s["bt"].gather(1, pos // ps).long()[:, None]
    at = (phys * c["Hkv"] + torch.arange(c["Hkv"], device=DEV)[:, None]) * ps + (pos % ps)[:, None]
    at = torch.where((pos < n)[:, None], at, pool.numel() - 1)
    old = torch.where((pos < n - L)[:, None], pool[at] * c["decay"], 0.0)
    pool[at] = old + w
    s["wp"].view(-1).copy_(pool[:-1])
    return out, s["wp"]


def _plain_evict(s):
    c = s["c"]
    B, Hkv, ps, keep = c["B"], c["Hkv"], c["ps"], c["keep"]
    n = s["cl"].long()[:, None, None]
    pos = torch.arange(s["max"], device=DEV)
    phys = s["bt"].gather(1, (pos // ps).expand(B, -1)).long().clamp_min(0)
    w = s["wp"][phys, :, pos % ps].transpose(1, 2)
    forced = (pos < c["S"]) | ((pos >= n - c["recent"]) & (pos < n))
    w = torch.where(pos < n, torch.where(forced, math.inf, w), -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.sort(order, dim=-1).values
    to = torch.arange(keep, device=DEV)
    head = torch.arange(Hkv, device=DEV)[:, None]
    src = s["bt"].gather(1, (kept // ps).reshape(B, -1)).view(B, Hkv, keep).long()
    dst = s["dst"].gather(1, (to // ps).expand(B, -1)).long()[:, None].expand(B, Hkv, keep)
    s["kp"][dst, head, to % ps] = s["kp"][src, head, kept % ps]
    s["vp"][dst, head, to % ps] = s["vp"][src, head, kept % ps]
    s["wp"][dst, head, to % ps] = s["wp"][src, head, kept % ps]
    s["kept"].copy_(kept)
    s["new_lens"].fill_(keep)
    return s["kept"], s["new_lens"], _view(s["kp"]), _view(s["vp"]), s["wp"]


# ---- the definitions, in 64 bits, one request at a time -------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "window": _exact_attention, "weights": _exact_attention, "evict": _exact_evict}[case["kind"]](s)


def _wide(pool):
    return pool.view(F8).float().double() if pool.dtype == torch.uint8 else pool.double()


def _exact_append(s):
    c = s["c"]
    kp, vp = _wide(s["kp"]), _wide(s["vp"])
    query = torch.zeros(s["query"].shape, dtype=torch.float64, device=DEV)
    half = c["R"] // 2
    unit = 0.02 if c["fp8"] else 1.0
    for b in range(c["B"]):
        x = s["qkv"][b].double().view(c["L"], -1, c["D"])
        table = s["cos_sin"][s["positions"][b].long()].double()
        turn = torch.complex(table[:, :half], table[:, half:])[:, None]
        page, off = s["slots"][b].long() // c["ps"], s["slots"][b].long() % c["ps"]
        for first, count, weight in ((0, c["Hq"], s["wq"]), (c["Hq"], c["Hkv"], s["wk"])):
            y = x[:, first : first + count].clone()
            if weight is not None:
                y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
            if c["inter"]:
                z = torch.complex(y[..., 0 : c["R"] : 2], y[..., 1 : c["R"] : 2]) * turn
                y[..., 0 : c["R"] : 2], y[..., 1 : c["R"] : 2] = z.real, z.imag
            else:
                z = torch.complex(y[..., :half], y[..., half : c["R"]]) * turn
                y[..., :half], y[..., half : c["R"]] = z.real, z.imag
            if first == 0:
                query[b] = y.transpose(0, 1)
            else:
                kp[page, :, off] = (y / unit).clamp(-448, 448) if c["fp8"] else y
        v = x[:, c["Hq"] + c["Hkv"] :]
        vp[page, :, off] = (v / unit).clamp(-448, 448) if c["fp8"] else v
    return query, kp, vp


def _exact_attention(s):
    c = s["c"]
    L, ps, unit = c["L"], c["ps"], 0.02 if c["fp8"] else 1.0
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    wp = s["wp"].double() if "wp" in s else None
    step = max(1, (1 << 26) // s["max"])
    for b, n in enumerate(s["cl"].tolist()):
        ids = torch.arange(n, device=DEV)
        if c["kind"] == "window":
            a, first = _visible(c, n)
            ids = ids[(ids < a) | (ids >= first)]
        page, off = s["bt"][b, ids // ps].long(), ids % ps
        for h in range(c["Hkv"]):
            k, v = (_wide(p[page, h, off]) * unit for p in (s["kp"], s["vp"]))
            got = torch.zeros(ids.shape, dtype=torch.float64, device=DEV)
            for g in range(h * G, (h + 1) * G):
                for i in range(0, L, step):
                    at = n - L + torch.arange(i, min(L, i + step), device=DEV)[:, None]
                    seen = ids <= at
                    if c["kind"] == "window":
                        seen &= (ids > at - c["W"]) | (ids < c["S"])
                    z = (s["q"][b, g, i : i + step].double() @ k.T) / math.sqrt(c["D"])
                    p = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
                    out[b, g, i : i + step] = p @ v
                    got += p.sum(0)
            if wp is not None:
                wp[page, h, off] = torch.where(ids < n - L, wp[page, h, off] * c["decay"], 0.0) + got
    return out if wp is None else (out, wp)


def _exact_evict(s):
    c = s["c"]
    kept = torch.zeros((c["B"], c["Hkv"], c["keep"]), dtype=torch.int64, device=DEV)
    kp, vp, wp = _wide(s["kp"]), _wide(s["vp"]), s["wp"].double()
    for b, n in enumerate(s["cl"].tolist()):
        pos = torch.arange(n, device=DEV)
        page, off = s["bt"][b, pos // c["ps"]].long(), pos % c["ps"]
        to = torch.arange(c["keep"], device=DEV)
        dpage, doff = s["dst"][b, to // c["ps"]].long(), to % c["ps"]
        free = n - c["S"] - c["recent"]
        for h in range(c["Hkv"]):
            w = wp[page, h, off]
            best = torch.argsort(-w[c["S"] : c["S"] + free], stable=True)[: c["keep"] - c["S"] - c["recent"]] + c["S"]
            kept[b, h] = torch.cat([pos[: c["S"]], best.sort().values, pos[n - c["recent"] :]])
            for pool in (kp, vp, wp):
                pool[dpage, h, doff] = pool[page[kept[b, h]], h, off[kept[b, h]]]
    return kept, torch.full((c["B"],), c["keep"], dtype=torch.int64, device=DEV), kp, vp, wp
