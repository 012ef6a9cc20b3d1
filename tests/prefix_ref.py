"""Inputs and plain 64-bit references of the decode behind shared prefixes."""
import math

import numpy as np
import torch

import q4_ref
from window_ref import F8, SCALES


def make(prefixes, lens, H_q, H_kv, L, D, ps, seed, pool="bf16", poison=True):
    """prefixes: (tokens, requests) of each; lens: every request's positions in all, the
    requests of the prefixes first. A prefix's whole pages are in its table alone (the
    requests' entries there are -1); what no row may see is NaN."""
    rng = np.random.default_rng(seed)
    plen_of = [n for n, k in prefixes for _ in range(k)] + [0] * (len(lens) - sum(k for _, k in prefixes))
    B, NP = len(lens), len(prefixes)
    width = max(1, max(-(-n // ps) for n in lens))
    pwidth = max(1, max(-(-n // ps) for n, _ in prefixes))
    own = [range(p // ps, -(-n // ps)) if n > p else range(0) for n, p in zip(lens, plen_of)]
    P = sum(-(-n // ps) for n, _ in prefixes) + sum(map(len, own)) + 3
    perm = rng.permutation(P).tolist()
    pt = torch.full((NP, pwidth), -1, dtype=torch.int32)
    bt = torch.full((B, width), -1, dtype=torch.int32)
    live = torch.zeros((P, ps), dtype=torch.bool)
    for i, (n, _) in enumerate(prefixes):
        for j in range(-(-n // ps)):
            pt[i, j] = perm.pop()
        at = torch.arange(n)
        live[pt[i, at // ps].long(), at % ps] = True
    for b, pages in enumerate(own):
        for j in pages:
            bt[b, j] = perm.pop()
        at = torch.arange(min(plen_of[b], lens[b]), lens[b])
        live[bt[b, at // ps].long(), at % ps] = True
    g = torch.Generator(device="cuda").manual_seed(seed)
    kp, vp = (torch.randn((P, H_kv, ps, D), generator=g, device="cuda") for _ in "kv")
    live = live.cuda()
    if pool == "bf16":
        kp, vp, bad = kp.to(torch.bfloat16), vp.to(torch.bfloat16), float("nan")
    elif pool == "e4m3":
        kp, vp = ((x / s).clamp(-448, 448).to(F8).view(torch.uint8) for x, s in zip((kp, vp), SCALES))
        bad = 0x7F
    else:
        kp, vp = (torch.from_numpy(q4_ref.quantise(x.to(torch.bfloat16).double().cpu().numpy())).cuda()
                  for x in (kp, vp))
        bad = 0xFF
    if poison:
        for x in (kp, vp):
            x.transpose(1, 2)[~live] = bad
    q = (torch.randn((B, H_q, L, D), generator=g, device="cuda") * 1.3).to(torch.bfloat16)
    starts = np.concatenate([[0], np.cumsum([k for _, k in prefixes])])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(query=q, key_pages=kp, value_pages=vp, block_table=bt.cuda(), context_lens=i32(lens), page_size=ps,
                prefix_table=pt.cuda(), prefix_lens=i32([n for n, _ in prefixes]), prefix_starts=i32(starts))


def _rows(pool, kind, page, off, shared):
    """Values [H, n, D] and the sizes of what is summed for them, as the calls round them."""
    x = pool[page, :, off].transpose(0, 1)
    if kind == "bf16":
        return x.double(), x.double().abs()
    if kind == "e4m3":
        return x.view(F8).float().double(), x.view(F8).float().double().abs()
    rows = x.cpu().numpy()
    c, s, m = q4_ref.parts(rows)
    if shared:
        v = torch.from_numpy((m + s * c).astype(np.float16).astype(np.float64)).cuda()
        return v, v.abs()
    sc = torch.from_numpy((s * c).astype(np.float16).astype(np.float64)).cuda()
    m = torch.from_numpy(m).cuda()
    return sc + m, sc.abs() + m.abs()


def reference(c, kind="bf16", group=None):
    """Per request (out, sum p |v|, largest scale * sum |q| |k|) in 64 bits. group: the
    prefix of each request (None: by prefix_starts)."""
    ps = c["page_size"]
    B, H_q, L, D = c["query"].shape
    H_kv = c["key_pages"].shape[1]
    starts, plens = c["prefix_starts"].tolist(), c["prefix_lens"].tolist()
    ks, vs = SCALES if kind == "e4m3" else (1.0, 1.0)
    got = []
    for b, n in enumerate(c["context_lens"].tolist()):
        p = next((i for i in range(len(plens)) if starts[i] <= b < starts[i + 1]), None)
        plen = min(n, plens[p]) if p is not None else 0
        j = torch.arange(n, device="cuda")
        parts = []
        if plen:
            parts.append((c["prefix_table"][p, j[:plen] // ps].long(), j[:plen] % ps, True))
        if n > plen:
            parts.append((c["block_table"][b, j[plen:] // ps].long(), j[plen:] % ps, False))
        q = c["query"][b].double()
        out, mag, size = torch.zeros_like(q), torch.zeros_like(q), 0.0
        if parts:
            k, v, ka, va = [], [], [], []
            for page, off, shared in parts:
                for pool, vals, sizes in ((c["key_pages"], k, ka), (c["value_pages"], v, va)):
                    x, a = _rows(pool, kind, page, off, shared)
                    vals.append(x)
                    sizes.append(a)
            k, v, ka, va = (torch.cat(x, 1).repeat_interleave(H_q // H_kv, 0) for x in (k, v, ka, va))
            see = j <= n - L + torch.arange(L, device="cuda")[:, None]
            scale = ks / math.sqrt(D)
            z = (q @ k.transpose(1, 2) * scale).masked_fill(~see, -math.inf)
            w = torch.softmax(z, -1).nan_to_num(0.0)
            out, mag = w @ v * vs, w @ va * vs
            size = float((q.abs() @ ka.transpose(1, 2)).max() * scale)
        got.append((out, mag, size))
    return got


def check(out, ref, kind, n_max, vmax):
    """Output rounding: half a step of bf16, 2^-8 of the value. The prefix's weights are
    rounded to bf16 for P . V, 2^-8 of each term (the others finer: two bf16, or f16 for
    codes, there in the prefix too, with 2^-25 a key where f16 is subnormal). Scores: D fp32 additions of
    truncated size, 2^-16 of scale * sum |q| |k|, on both sides of the quotient. The sums:
    n roundings; the merge: three more of 2^-22 each (ex2)."""
    for b, (r, mag, size) in enumerate(ref):
        got = out[b].double()
        assert torch.isfinite(got).all(), f"request {b}"
        tol = r.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + size * 2.0 ** -15 + n_max * 2.0 ** -24 + 2.0 ** -20) + 1e-30
        if kind != "bf16":
            tol = tol + n_max * 2.0 ** -25 * vmax
        err = (got - r).abs()
        assert torch.all(err <= tol), (b, float((err / tol).max()))
