"""Inputs and plain 64-bit references of the sliding-window and weight tests,
and the tolerances that follow from the kernels' roundings."""
import math

import torch

F8 = torch.float8_e4m3fn
SCALES = (0.03, 0.02)


def seen_rows(n, L, W, S, causal=True):
    """[L, n] truth values: which keys each row sees. W None: no window."""
    p = (n - L + torch.arange(L, device="cuda"))[:, None]
    j = torch.arange(n, device="cuda")[None]
    if not causal:
        return (j >= 0).expand(L, n)
    see = j <= p
    return see if W is None else see & ((j > p - W) | (j < S))


def make(lens, H_q, H_kv, L, D, ps, seed, W=None, S=0, fp8=False, poison=True, max_pages=None):
    """A batch whose pages no row sees have table entry -1 (window) and whose
    slots that no row sees hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    need = []
    for n in lens:
        see = seen_rows(n, L, W, S).any(0) if n else torch.zeros(0, dtype=torch.bool)
        pages = set((see.nonzero().flatten() // ps).tolist()) if W is not None else set(range(-(-n // ps)))
        need.append(sorted(pages))
    P = sum(len(x) for x in need) + 3
    perm = torch.randperm(P, generator=g, device="cuda").tolist()
    width = max_pages or max(1, max(-(-n // ps) for n in lens))
    bt = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(need):
        for j in x:
            bt[b, j] = perm[at]
            at += 1
    kp, vp = (torch.randn((P, H_kv, ps, D), generator=g, device="cuda") for _ in "kv")
    if fp8:
        kp, vp = ((x / s).clamp(-448, 448).to(F8).view(torch.uint8) for x, s in zip((kp, vp), SCALES))
    else:
        kp, vp = kp.to(torch.bfloat16), vp.to(torch.bfloat16)
    if poison:
        live = torch.zeros((P, ps), dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            if n:
                j = seen_rows(n, L, W, S).any(0).nonzero().flatten()
                live[bt[b].cuda()[j // ps].long(), j % ps] = True
        bad = 0x7F if fp8 else float("nan")
        for x in (kp, vp):
            x.transpose(1, 2)[~live] = bad
    q = (torch.randn((B, H_q, L, D), generator=g, device="cuda") * 1.3).to(torch.bfloat16)
    return dict(query=q, key_pages=kp, value_pages=vp, block_table=bt.cuda(),
                context_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), page_size=ps)


def reference(c, W=None, S=0, fp8=False, causal=True):
    """Per request: (out [H_q, L, D], sum p |v|, largest scale * sum |q| |k|,
    weights [H_kv, n]), in 64 bits."""
    ps = c["page_size"]
    B, H_q, L, D = c["query"].shape
    H_kv = c["key_pages"].shape[1]
    scale = 1 / math.sqrt(D)
    got = []
    for b, n in enumerate(c["context_lens"].tolist()):
        q = c["query"][b].double()
        out, mag = torch.zeros_like(q), torch.zeros_like(q)
        weights = torch.zeros((H_kv, n), dtype=torch.float64, device="cuda")
        size = 0.0
        if n:
            see = seen_rows(n, L, W, S, causal)
            j = see.any(0).nonzero().flatten()
            if len(j):
                page = c["block_table"][b, j // ps].long()
                k, v = (x[page, :, j % ps].transpose(0, 1) for x in (c["key_pages"], c["value_pages"]))
                if fp8:
                    k, v = k.view(F8).float().double() * SCALES[0], v.view(F8).float().double() * SCALES[1]
                k, v = (x.double().repeat_interleave(H_q // H_kv, 0) for x in (k, v))
                z = (q @ k.transpose(1, 2) * scale).masked_fill(~see[:, j], -math.inf)
                p = torch.softmax(z, -1).nan_to_num(0.0)       # a row that sees nothing
                out, mag = p @ v, p @ v.abs()
                size = float((q.abs() @ k.abs().transpose(1, 2)).max() * scale)
                weights[:, j] = p.view(H_kv, -1, L, len(j)).sum((1, 2))
        got.append((out, mag, size, weights))
    return got


def check_out(out, ref, fp8, n_max, vmax=448 * SCALES[1]):
    """Output rounding: half a step of bf16, 2^-8 of the value. Weights rounded
    for P . V: bf16, 2^-8 of each term, so 2^-8 sum p |v| (e4m3 pools: f16,
    2^-11, twice: the weights and a warp's O / l, with 2^-25 per key where f16
    is subnormal). Scores: D fp32 additions of truncated size, 2^-16 of
    scale * sum |q| |k|, on both sides of the quotient. The sum l: n roundings."""
    for b, (r, mag, size, _) in enumerate(ref):
        got = out[b].double()
        assert torch.isfinite(got).all(), f"request {b}"
        p_err = 2.0 ** -10 if fp8 else 2.0 ** -8
        tol = r.abs() * 2.0 ** -8 + mag * (p_err + size * 2.0 ** -15 + n_max * 2.0 ** -24) + 1e-30
        if fp8:
            tol = tol + n_max * 2.0 ** -25 * vmax
        err = (got - r).abs()
        assert torch.all(err <= tol), (b, float((err / tol).max()))
