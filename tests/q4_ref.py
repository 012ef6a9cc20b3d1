"""The 4-bit rows in numpy, from their definition, and inputs and 64-bit references
of the attention over them."""
import math

import numpy as np
import torch

from window_ref import seen_rows

GROUP, ROW, D = 32, 80, 128


def quantise(x):
    """x [..., 128] float64 (bf16 values) -> rows [..., 80] uint8."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        y = np.clip(x, -448.0, 448.0).astype(np.float16).reshape(*x.shape[:-1], D // GROUP, GROUP)
        m = y.min(-1, keepdims=True)
        step = ((y.max(-1, keepdims=True).astype(np.float32) - m.astype(np.float32)) /
                np.float32(15)).astype(np.float16)
        ratio = (y.astype(np.float64) - m) / step.astype(np.float64)
        code = np.where(step > 0, np.clip(np.rint(ratio), 0, 15), 0)
    code = np.nan_to_num(code).astype(np.uint8).reshape(*x.shape)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    parts = np.concatenate([step, m], -1).reshape(*x.shape[:-1], 2 * D // GROUP)
    return np.concatenate([packed, np.ascontiguousarray(parts).view(np.uint8)], -1)


def parts(rows):
    """rows [..., 80] uint8 (numpy) -> codes [..., 128], steps and least values spread to
    [..., 128], float64."""
    code = np.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).reshape(*rows.shape[:-1], D)
    p = np.ascontiguousarray(rows[..., 64:]).view(np.float16).reshape(*rows.shape[:-1], D // GROUP, 2)
    s, m = (np.repeat(p[..., i].astype(np.float64), GROUP, -1) for i in range(2))
    return code.astype(np.float64), s, m


def dense_values(rows):
    """What the read-back gives: m + s c in fp32, then bf16 (as float64)."""
    c, s, m = parts(rows)
    f = torch.from_numpy((m + s * c).astype(np.float32))
    return f.to(torch.bfloat16).double().numpy()


def make(lens, H_q, H_kv, L, ps, seed, poison=True, std=1.0):
    """A batch over 4-bit pools; slots behind a context have NaN groups."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    counts = [-(-n // ps) for n in lens]
    P = sum(counts) + 3
    perm = rng.permutation(P)
    bt = np.full((B, max(1, max(counts))), -1, np.int32)
    at = 0
    for b, k in enumerate(counts):
        bt[b, :k] = perm[at:at + k]
        at += k
    pools = []
    for _ in "kv":
        x = rng.standard_normal((P, H_kv, ps, D)) * std
        x[..., :3] *= 5
        rows = quantise(torch.from_numpy(x).to(torch.bfloat16).double().numpy())
        if poison:
            live = np.zeros((P, ps), bool)
            for b, n in enumerate(lens):
                j = np.arange(n)
                live[bt[b, j // ps], j % ps] = True
            rows.transpose(0, 2, 1, 3)[~live] = 0xFF      # f16 0xFFFF is a NaN
        pools.append(torch.from_numpy(rows).cuda())
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn((B, H_q, L, D), generator=g, device="cuda") * 1.3).to(torch.bfloat16)
    return dict(query=q, key_pages=pools[0], value_pages=pools[1], block_table=torch.from_numpy(bt).cuda(),
                context_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), page_size=ps)


def reference(c, copied=False, causal=True, scale=None):
    """As window_ref.reference, with the roundings that the calls document left in: s c to
    f16 (decode), or keys to bf16 and values to f16 (copied: prefill). The magnitudes are those of
    s c and m apart, as the decode sums them."""
    ps = c["page_size"]
    B, H_q, L, _ = c["query"].shape
    H_kv = c["key_pages"].shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    got = []
    for b, n in enumerate(c["context_lens"].tolist()):
        q = c["query"][b].double()
        out, mag, size = torch.zeros_like(q), torch.zeros_like(q), 0.0
        if n:
            j = torch.arange(n, device="cuda")
            page = c["block_table"][b, j // ps].long()
            vals, sizes = [], []
            for pool in (c["key_pages"], c["value_pages"]):
                rows = pool[page, :, j % ps].transpose(0, 1).cpu().numpy()
                code, s, m = parts(rows)
                if copied:
                    v = (m + s * code).astype(np.float32).astype(np.float16).astype(np.float64) if vals \
                        else dense_values(rows)
                    w = np.abs(v)
                else:
                    sc = (s * code).astype(np.float16).astype(np.float64)
                    v, w = sc + m, np.abs(sc) + np.abs(m)
                vals.append(torch.from_numpy(v).cuda().repeat_interleave(H_q // H_kv, 0))
                sizes.append(torch.from_numpy(w).cuda().repeat_interleave(H_q // H_kv, 0))
            see = seen_rows(n, L, None, 0, causal)
            z = (q @ vals[0].transpose(1, 2) * scale).masked_fill(~see, -math.inf)
            p = torch.softmax(z, -1).nan_to_num(0.0)
            out, mag = p @ vals[1], p @ sizes[1]
            size = float((q.abs() @ sizes[0].transpose(1, 2)).max() * scale)
        got.append((out, mag, size, None))
    return got
