"""Cases, plain forms and calls of the operators that cut the bytes a decode reads.

Three kinds of case, each one pass of a serving step's work on one layer:

  cache    new K/V rows quantised to 4 bits as they are written into the pages, and the requests' cached rows read back
  attend   attention over 4-bit pages
  prefix   decode of a batch whose requests share long prefixes, each prefix attended to once for all of them

A row of a 4-bit pool is 80 bytes: the codes of 128 elements (element d in byte d // 2, even d in the low half), then for
each group of 32 elements the step and the least value as 16-bit floats. A code c stands for least + step * c.

`own` chooses between the plain form (torch operations in 32 bits) and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
SCALE8 = 0.02
GROUP = 32
ROW4 = 80


def listed():
    return [
        # one new token of one request, its short context read back: the latency of the two calls
        dict(name="cache_1_token", kind="cache", B=1, L=1, Hkv=4, ps=16, lo=300, hi=300),
        # a decode batch's tokens, and the ragged contexts for a consumer of dense rows
        dict(name="cache_b32", kind="cache", B=32, L=1, Hkv=4, ps=16, lo=128, hi=4096),
        # prompts of an odd length, written and read back whole
        dict(name="cache_prompt_4x2047", kind="cache", B=4, L=2047, Hkv=8, ps=16, lo=2047, hi=4099),
        # one request: the latency of a single decode, 7 query heads per KV head
        dict(name="attend_b1", kind="attend", B=1, L=1, Hq=28, Hkv=4, ps=16, lo=5001, hi=5001),
        # a ragged decode batch
        dict(name="attend_b32_gqa7", kind="attend", B=32, L=1, Hq=28, Hkv=4, ps=16, lo=128, hi=4096),
        # a large decode batch with large pages
        dict(name="attend_b64_ps128", kind="attend", B=64, L=1, Hq=32, Hkv=8, ps=128, lo=64, hi=8192),
        # long contexts
        dict(name="attend_long_b8", kind="attend", B=8, L=1, Hq=32, Hkv=8, ps=16, lo=16384, hi=32768),
        # prefill chunks after ragged prefixes
        dict(name="attend_prefill_4x512", kind="attend", B=4, L=512, Hq=32, Hkv=8, ps=16, lo=512, hi=2560),
        # a few requests over one system prompt
        dict(name="prefix_b8", kind="prefix", B=8, L=1, Hq=28, Hkv=4, D=128, ps=16, NP=1, plo=2048, phi=2048, lo=16, hi=256, pool="bf16"),
        # a ragged decode batch over one long document
        dict(name="prefix_b32_gqa7", kind="prefix", B=32, L=1, Hq=28, Hkv=4, D=128, ps=16, NP=1, plo=16384, phi=16384, lo=64, hi=1024, pool="bf16"),
        # a large batch over three prefixes of different lengths, e4m3 pools with large pages
        dict(name="prefix_3_b64_e4m3", kind="prefix", B=64, L=1, Hq=32, Hkv=8, D=128, ps=128, NP=3, plo=3000, phi=20000, lo=64, hi=2048, pool="e4m3"),
        # drafts of four tokens over one prefix, 4-bit pools
        dict(name="prefix_draft4_b16_q4", kind="prefix", B=16, L=4, Hq=32, Hkv=8, D=128, ps=16, NP=1, plo=8192, phi=8192, lo=100, hi=1500, pool="q4"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["cache", "attend", "attend", "prefix", "prefix"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = min(Hkv * rng.choice([1, 2, 3, 4, 7, 8]), 32 // Hkv * Hkv)
    ps = rng.choice([1, 4, 16, 16, 32, 64, 128, 256])
    if kind == "cache":
        B = _log(rng, 1, 32)
        L = rng.choice([1, _log(rng, 1, max(1, 8000 // B))])
        lo = L + rng.choice([0, _log(rng, 1, max(2, 12000 // B))])
        return dict(kind=kind, B=B, L=L, Hkv=Hkv, ps=ps, lo=lo, hi=lo + _log(rng, 1, max(2, 12000 // B)))
    if kind == "attend":
        if rng.random() < 0.75:
            L = rng.choice([1, 1, 1, 2, 3, 5])
            lo = L + _log(rng, 1, 16000)
            hi = lo + _log(rng, 1, 16000)
            B = _log(rng, 1, max(1, min(64, 1500000 // (Hkv * hi))))
        else:
            B = _log(rng, 1, 4)
            L = _log(rng, 33, 1200 // B)
            lo = L + _log(rng, 1, 800)
            hi = lo + _log(rng, 1, 800)
        return dict(kind=kind, B=B, L=L, Hq=Hq, Hkv=Hkv, ps=ps, lo=lo, hi=hi)
    pool = rng.choice(["bf16", "bf16", "e4m3", "q4"])
    B = _log(rng, 2, 64)
    L = rng.choice([1, 1, 1, 2, 4])
    NP = rng.choice([1, 1, 1, 2, 4])
    plo = _log(rng, 100, min(12000, 1000000 // (B * L)))
    lo = _log(rng, 1, 1000)
    return dict(kind=kind, B=B, L=L, Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128]) if pool == "bf16" else 128, ps=ps, NP=min(NP, B), plo=plo,
                phi=plo + rng.choice([0, _log(rng, 1, plo)]), lo=lo, hi=lo + _log(rng, 1, 1500), pool=pool)


def _spread(lo, hi, n):
    """n lengths over [lo, hi], evenly over their logarithm."""
    if n == 1:
        return [hi]
    return [min(hi, max(lo, int(round(lo * (hi / lo) ** (i / (n - 1)))))) for i in range(n)]


def _prefixes(c):
    """Lengths of the prefixes, and how many requests share each: the first ones more."""
    shares = [c["B"] // c["NP"] + (1 if i < c["B"] % c["NP"] else 0) for i in range(c["NP"])]
    return _spread(c["plo"], c["phi"], c["NP"]), shares


def work(c):
    Hkv, L, B = c["Hkv"], c["L"], c["B"]
    if c["kind"] == "cache":
        new, held = B * L, sum(_spread(c["lo"], c["hi"], B))
        return {"bytes": new * (Hkv * 2 * (256 + ROW4) + 4) + held * Hkv * 2 * (ROW4 + 256), "flops": (new * 6 + held * 2) * Hkv * 2 * 128}
    rows = B * c["Hq"] * L
    if c["kind"] == "attend":
        lens = _spread(c["lo"], c["hi"], B)
        pairs = sum(sum(n - L + i + 1 for i in range(L)) for n in lens) * c["Hq"]
        return {"bytes": rows * 512 + sum(lens) * Hkv * 2 * ROW4, "flops": 4 * pairs * 128}
    D = c["D"]
    row = {"bf16": 2 * D, "e4m3": D, "q4": ROW4}[c["pool"]]
    plens, shares = _prefixes(c)
    own_lens = _spread(c["lo"], c["hi"], B)
    own_pairs = sum(n * L - L * (L - 1) // 2 if n >= L else n * (n + 1) // 2 for n in own_lens)
    pairs = sum(p * k * L for p, k in zip(plens, shares)) + own_pairs
    return {"bytes": rows * 4 * D + (sum(plens) + sum(own_lens)) * Hkv * 2 * row, "flops": 4 * pairs * c["Hq"] * D}


# ---- inputs ---------------------------------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(torch.bfloat16)


def _rows(g, shape, std=1.0):
    """K or V rows: normal, a few elements of the head larger than the others in every token, as keys have them."""
    big = torch.ones(shape[-1], device=DEV)
    big[torch.randperm(shape[-1], generator=g, device=DEV)[: shape[-1] // 32]] = 4.0
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * big * std).to(torch.bfloat16)


def _pool(g, shape, kind):
    x = _rows(g, shape)
    if kind == "bf16":
        return x
    if kind == "e4m3":
        return (x.float() / SCALE8).clamp(-448, 448).to(F8).view(torch.uint8)
    out = torch.empty((*shape[:-1], ROW4), dtype=torch.uint8, device=DEV)
    for a, b in zip(x.split(4096), out.split(4096)):
        b.copy_(_quantised(a))
    return out


def _pages(g, counts, spare=3):
    """One row of distinct physical pages for each count, -1 behind them, and the number of pages in the pool."""
    total = sum(counts) + spare
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(counts), max(1, max(counts))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, k in enumerate(counts):
        table[i, :k] = perm[at : at + k]
        at += k
    return table, total


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    ps, Hkv, B, L = c["ps"], c["Hkv"], c["B"], c["L"]
    lens = _spread(c["lo"], c["hi"], B)
    lens = [lens[i] for i in torch.randperm(B, generator=g, device=DEV).tolist()]
    if c["kind"] == "prefix":
        s["plens"], shares = _prefixes(c)
        s["group"] = [p for p, k in enumerate(shares) for _ in range(k)]
        s["prefix_lens"] = torch.tensor(s["plens"], dtype=torch.int32, device=DEV)
        s["starts"] = [sum(shares[:p]) for p in range(c["NP"] + 1)]
        s["prefix_starts"] = torch.tensor(s["starts"], dtype=torch.int32, device=DEV)
        lens = [n + s["plens"][p] for n, p in zip(lens, s["group"])]
        # a prefix's whole pages are shared; its last tokens lie in a page of each request
        shared = [p // ps for p in s["plens"]]
        own_counts = [-(-n // ps) - shared[p] for n, p in zip(lens, s["group"])]
        rows, P = _pages(g, [-(-p // ps) for p in s["plens"]] + own_counts)
        s["prefix_table"] = rows[: c["NP"], : max(1, max(-(-p // ps) for p in s["plens"]))].contiguous()
        table = torch.full((B, max(-(-n // ps) for n in lens)), -1, dtype=torch.int32, device=DEV)
        for b, p in enumerate(s["group"]):
            table[b, : shared[p]] = rows[p, : shared[p]]
            table[b, shared[p] : shared[p] + own_counts[b]] = rows[c["NP"] + b, : own_counts[b]]
    else:
        table, P = _pages(g, [-(-n // ps) for n in lens])
    s["bt"] = table.contiguous()
    s["cl"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["max"] = max(lens)
    if c["kind"] == "cache":
        s["k"], s["v"] = (_rows(g, (B, Hkv, L, 128)) for _ in range(2))
        t = s["cl"].long()[:, None] - L + torch.arange(L, device=DEV)
        s["slots"] = (table.gather(1, t // ps) * ps + t % ps).to(torch.int32)
        s["kp"], s["vp"] = (_pool(g, (P, Hkv, ps, 128), "q4") for _ in range(2))
        s["kd"], s["vd"] = (torch.zeros((B, Hkv, s["max"], 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        return s
    D = c.get("D", 128)
    pool = c.get("pool", "q4")
    s["kp"], s["vp"] = (_pool(g, (P, Hkv, ps, D), pool) for _ in range(2))
    s["q"] = _normal(g, (B, c["Hq"], L, D), 1.0)
    s["out"] = torch.empty_like(s["q"])
    if own:
        s["ws"] = _workspace(s)
    return s


def _workspace(s):
    import paged_kv_attention_06_gb300 as pa

    c = s["c"]
    B, Hq, L, D = s["q"].shape
    shape = pa.pa_shape(B, Hq, c["Hkv"], D, L, s["kp"].shape[0], s["bt"].shape[1])
    if c["kind"] == "attend":
        need = pa.pa_attention_q4_workspace_bytes(shape, s["max"])
    else:
        f = {"bf16": pa.pa_decode_prefix_workspace_bytes, "e4m3": pa.pa_decode_prefix_fp8_workspace_bytes, "q4": pa.pa_decode_prefix_q4_workspace_bytes}[c["pool"]]
        need = f(shape, c["ps"], c["NP"], max(s["plens"]))
    return torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)


# ---- one pass -------------------------------------------------------------------------------------------------------


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import paged_kv_attention_06_gb300 as pa

    c = s["c"]
    if c["kind"] == "cache":
        pa.pa_append_kv_q4(s["k"], s["v"], s["kp"], s["vp"], s["slots"], c["ps"])
        return pa.pa_gather_kv_q4(s["kp"], s["vp"], s["bt"], s["cl"], c["ps"], s["max"], key_dense=s["kd"], value_dense=s["vd"])
    if c["kind"] == "attend":
        return pa.pa_attention_q4(s["q"], s["kp"], s["vp"], s["bt"], s["cl"], c["ps"], out=s["out"], max_context_len=s["max"], workspace=s["ws"])
    f = {"bf16": pa.pa_decode_prefix, "e4m3": pa.pa_decode_prefix_fp8, "q4": pa.pa_decode_prefix_q4}[c["pool"]]
    scales = (SCALE8, SCALE8) if c["pool"] == "e4m3" else ()
    return f(s["q"], s["kp"], s["vp"], s["bt"], s["cl"], c["ps"], *scales, prefix_table=s["prefix_table"], prefix_lens=s["prefix_lens"],
             prefix_starts=s["prefix_starts"], max_prefix_len=max(s["plens"]), out=s["out"], max_context_len=s["max"], workspace=s["ws"])


def _plain(s):
    return {"cache": _plain_cache, "attend": _plain_attend, "prefix": _plain_prefix}[s["c"]["kind"]](s)


def _quantised(x):
    """Rows [..., 128] bf16 as rows of a 4-bit pool [..., 80] uint8."""
    y = x.float().clamp(-448.0, 448.0).half().unflatten(-1, (4, GROUP))
    least = y.amin(-1, keepdim=True)
    span = y.amax(-1, keepdim=True).float() - least.float()
    step = (span / torch.full_like(span, 15.0)).half()
    # in 64 bits: a quotient next to a half would round to it in 32
    code = ((y.double() - least.double()) / step.double().clamp_min(1e-30)).round().clamp(0, 15)
    code = torch.where(step > 0, code, 0.0).to(torch.uint8).flatten(-2)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    parts = torch.cat([step, least], -1).flatten(-2)
    return torch.cat([packed, parts.view(torch.uint8)], -1)


def _values(rows):
    """Rows [..., 80] of a 4-bit pool as the values they stand for, [..., 128] in 32 bits."""
    code = torch.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).flatten(-2).unflatten(-1, (4, GROUP))
    parts = rows[..., 64:].contiguous().view(torch.float16).unflatten(-1, (4, 2)).float()
    return (parts[..., 1:] + parts[..., :1] * code.float()).flatten(-2)


def _wide(pool, rows):
    if pool == "q4":
        return _values(rows)
    return rows.view(F8).float() * SCALE8 if pool == "e4m3" else rows.float()


def _plain_cache(s):
    c = s["c"]
    ps = c["ps"]
    slot = s["slots"].long().view(-1)
    for pool, new in ((s["kp"], s["k"]), (s["vp"], s["v"])):
        pool[slot // ps, :, slot % ps] = _quantised(new).transpose(1, 2).reshape(-1, c["Hkv"], ROW4)
    pos = torch.arange(s["max"], device=DEV)
    phys = s["bt"].gather(1, (pos // ps).expand(c["B"], -1)).long().clamp_min(0)
    there = (pos < s["cl"][:, None])[:, None, :, None]
    for pool, dense in ((s["kp"], s["kd"]), (s["vp"], s["vd"])):
        dense.copy_(torch.where(there, _values(pool[phys, :, pos % ps]).transpose(1, 2), dense.float()))
    return s["kd"], s["vd"]


def _gathered(s, table, length):
    """K and V at positions 0 .. length - 1 of each of the table's rows: [N, Hkv, length, D] in 32 bits."""
    c = s["c"]
    pos = torch.arange(length, device=DEV)
    phys = table.gather(1, (pos // c["ps"]).expand(table.shape[0], -1)).long().clamp_min(0)
    return [_wide(c.get("pool", "q4"), p[phys, :, pos % c["ps"]]).transpose(1, 2) for p in (s["kp"], s["vp"])]


def _softmax_times(s, z, v):
    """The rows' attention from masked scores z [B, Hkv, G, L, n] and values v [B, Hkv, n, D]."""
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp_min(-1e30))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    s["out"].copy_((p.flatten(2, 3) @ v).view(s["out"].shape))
    return s["out"]


def _scores(s, k):
    c = s["c"]
    q = s["q"].float().view(c["B"], c["Hkv"], -1, s["q"].shape[3])
    return ((q @ k.transpose(-1, -2)) * s["q"].shape[3] ** -0.5).view(c["B"], c["Hkv"], -1, c["L"], k.shape[-2])


def _last(s):
    """Each row's last visible position, [B, L]."""
    return s["cl"].long()[:, None] - s["c"]["L"] + torch.arange(s["c"]["L"], device=DEV)


def _plain_attend(s):
    k, v = _gathered(s, s["bt"], s["max"])
    seen = torch.arange(s["max"], device=DEV) <= _last(s)[:, :, None]
    return _softmax_times(s, _scores(s, k).masked_fill(~seen[:, None, None], -math.inf), v)


def _plain_prefix(s):
    c = s["c"]
    B, Hkv, L, D = c["B"], c["Hkv"], c["L"], c["D"]
    ps = c["ps"]
    groups = list(enumerate(zip(s["starts"], s["starts"][1:])))
    plen = s["prefix_lens"].long()[(torch.arange(B, device=DEV)[:, None] >= s["prefix_starts"][1:]).sum(1)]
    last = _last(s)
    # the prefixes, each for the rows of its requests; a request's own tokens behind it
    longest = max(s["plens"])
    pk, pv = _gathered(s, s["prefix_table"], longest)
    q = s["q"].float().view(B, Hkv, -1, D)
    at = torch.arange(longest, device=DEV)
    pz = torch.empty((B, Hkv, q.shape[2], longest), device=DEV)
    for p, (a, b) in groups:
        pz[a:b] = (q[a:b].transpose(0, 1).flatten(1, 2) @ pk[p].transpose(-1, -2)).view(Hkv, -1, q.shape[2], longest).transpose(0, 1) * D**-0.5
    pz = pz.view(B, Hkv, -1, L, longest).masked_fill(~((at < plen[:, None])[:, None] & (at <= last[:, :, None]))[:, None, None], -math.inf)
    rest = int(c["hi"])
    pos = plen[:, None] + torch.arange(rest, device=DEV)
    inside = pos < s["cl"][:, None]
    pos = torch.where(inside, pos, s["cl"].long()[:, None] - 1)
    phys = s["bt"].gather(1, pos // ps).long().clamp_min(0)
    k, v = (_wide(c["pool"], x[phys, :, pos % ps]).transpose(1, 2) for x in (s["kp"], s["vp"]))
    seen = inside[:, None] & (pos[:, None] <= last[:, :, None])
    z = _scores(s, k).masked_fill(~seen[:, None, None], -math.inf)
    top = torch.maximum(pz.amax(-1), z.amax(-1)).clamp_min(-1e30)[..., None]
    pe, e = torch.exp(pz - top).flatten(2, 3), torch.exp(z - top).flatten(2, 3)
    out = e @ v
    for p, (a, b) in groups:
        out[a:b] += (pe[a:b].transpose(0, 1).flatten(1, 2) @ pv[p]).view(Hkv, -1, q.shape[2], D).transpose(0, 1)
    out /= (pe.sum(-1, keepdim=True) + e.sum(-1, keepdim=True)).clamp_min(1e-30)
    s["out"].copy_(out.view(s["out"].shape))
    return s["out"]


# ---- the definitions, in 64 bits, one request at a time -------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_cache(s) if case["kind"] == "cache" else _exact_attention(s)


def _exact_values(rows):
    """What rows of a 4-bit pool stand for, in 64 bits, element by element."""
    d = torch.arange(128, device=DEV)
    code = (rows[..., d // 2].int() >> (4 * (d % 2)).int()) & 15
    parts = rows[..., 64:].contiguous().view(torch.float16).double()
    return parts[..., 2 * (d // GROUP) + 1] + parts[..., 2 * (d // GROUP)] * code.double()


def _exact_rows(s, page, h, off):
    c = s["c"]
    if c.get("pool", "q4") == "q4":
        return [_exact_values(p[page, h, off]) for p in (s["kp"], s["vp"])]
    return [p[page, h, off].view(F8).float().double() * SCALE8 if c["pool"] == "e4m3" else p[page, h, off].double() for p in (s["kp"], s["vp"])]


def _exact_cache(s):
    c = s["c"]
    got = []
    for pool, new in ((s["kp"], s["k"]), (s["vp"], s["v"])):
        dense = torch.zeros(s["kd"].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["cl"].tolist()):
            pos = torch.arange(n, device=DEV)
            dense[b, :, :n] = _exact_values(pool[s["bt"][b, pos // c["ps"]].long(), :, pos % c["ps"]]).transpose(0, 1)
            x = new[b].double().clamp(-448, 448).view(c["Hkv"], c["L"], -1, GROUP)
            low, high = x.min(-1, keepdim=True).values.half().double(), x.max(-1, keepdim=True).values
            step = ((high - low) / 15).half().double()
            code = torch.clamp(torch.round((x - low) / step), 0, 15)
            dense[b, :, n - c["L"] : n] = torch.where(step > 0, low + step * code, low).view(c["Hkv"], c["L"], 128)
        got.append(dense)
    return got


def _exact_attention(s):
    c = s["c"]
    L, ps, G = c["L"], c["ps"], c["Hq"] // c["Hkv"]
    D = s["q"].shape[3]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["cl"].tolist()):
        ids = torch.arange(n, device=DEV)
        page = s["bt"][b, ids // ps].long()
        if c["kind"] == "prefix":
            p = s["group"][b]
            shared = ids < s["plens"][p]
            page[shared] = s["prefix_table"][p, ids[shared] // ps].long()
        at = n - L + torch.arange(L, device=DEV)[:, None]
        for h in range(c["Hkv"]):
            k, v = _exact_rows(s, page, h, ids % ps)
            z = (s["q"][b, h * G : (h + 1) * G].double() @ k.T) / math.sqrt(D)
            out[b, h * G : (h + 1) * G] = torch.softmax(z.masked_fill(ids > at, -math.inf), -1) @ v
    return out
