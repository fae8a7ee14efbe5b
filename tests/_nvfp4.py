"""Seeded NVFP4 caches and a 64-bit reference for the tests of the operators over them."""
import math

import numpy as np
import torch

import _attn
from oracle import formats

PAGE, BLOCK, DIM, GROUP = 64, 128, 128, 16
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def quantize(x, outer=1.0):
    """Bytes of codes and scales of bf16 rows, by the oracle (outer: a power of two)."""
    bits = (x.float() / outer).to(torch.bfloat16).contiguous().view(torch.int16).numpy().view(np.uint16)
    payload, scale = formats.nvfp4_quantize(bits.reshape(-1, DIM))
    return (torch.from_numpy(np.ascontiguousarray(payload)).reshape(*x.shape[:-1], DIM // 2),
            torch.from_numpy(np.ascontiguousarray(scale)).reshape(*x.shape[:-1], DIM // GROUP))


def plane(rows, seed, spread=0):
    """Codes of every value, scales of N(0, 1) rows; spread: scales of every size instead, a
    group's exponent in [-spread, spread] of E4M3's."""
    g = torch.Generator().manual_seed(seed)
    payload = torch.randint(0, 256, (rows, DIM // 2), generator=g).to(torch.uint8)
    s = 0.2 + 0.2 * torch.rand((rows, DIM // GROUP), generator=g)
    if spread:
        s = s * torch.exp2(torch.randint(-spread, spread + 1, s.shape, generator=g).float())
    return payload, s.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)


def values64(p, rows, outer=1.0):
    payload, scale = p[0][rows], p[1][rows].contiguous().view(torch.float8_e4m3fn).double()
    codes = torch.stack([GRID[(payload & 15).long()], GRID[(payload >> 4).long()]], -1).reshape(-1, DIM // GROUP, GROUP)
    return (codes * scale[..., None] * outer).reshape(-1, DIM)


def make(lens, kv_heads, seed, pads=(), garbage=True, max_pages=None, spread=0):
    """lens: [R][P].  Every code and scale that no row sees is NaN when garbage is set."""
    c = _attn.make("bf16", lens, kv_heads, seed, pads, False, max_pages)
    rows = c.num_pages * kv_heads * PAGE
    c.dtype = "nvfp4"
    c.k, c.v = plane(rows, seed + 1), plane(rows, seed + 2, spread)
    seen = torch.zeros(rows, dtype=torch.bool)
    for r, row in enumerate(lens):
        if r in pads:
            continue
        n = min(max(0, max(row)), c.page_table.shape[1] * PAGE)
        pages = c.page_table[int(c.slot_ids[r])].tolist()
        for h in range(kv_heads):
            at = _attn.token_rows(pages, n, h, kv_heads)
            seen[at] = True
        if garbage:
            c.page_table[int(c.slot_ids[r]), -(-n // PAGE):] = -1
    if garbage:
        for payload, scale in (c.k, c.v):
            payload[~seen] = 0xf7
            scale[~seen] = 0x7f
    return c


def reference(c, q, sm_scale, block_ids=None, lists=0, k_outer=1.0, v_outer=1.0):
    """out, lse in 64 bits and the bounds on their errors that the kernels' roundings allow:
    scores: 128 exact products summed in fp32 (the tensor cores may truncate: 2^-23 a step), a
    query element off by 2^-32 of its row's largest, two more roundings: e_s;
    lse: e_s, ex2's 2^-22 and the sum's roundings;
    out: each weight off by e_s and 2^-11 (f16) or 2^-31 of the row's largest weight (f16's
    subnormals), against sum w |v|; then one bf16 rounding of the result."""
    R, P, Hq, _ = q.shape
    out = torch.zeros((R, P, Hq, DIM), dtype=torch.float64)
    lse = torch.full((R, P, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    q64 = q.double()
    for r in range(R):
        slot = int(c.slot_ids[r])
        if not 0 <= slot < c.page_table.shape[0]:
            continue
        pages = c.page_table[slot].tolist()
        longest = min(max(c.row_lens[r].tolist()), len(pages) * PAGE)
        if longest <= 0:
            continue
        for h in range(c.kv_heads):
            rows = _attn.token_rows(pages, longest, h, c.kv_heads)
            page = rows // (PAGE * c.kv_heads)
            good = (page >= 0) & (page < c.num_pages)
            at = rows.clamp(0, len(c.k[0]) - 1)
            K, V = values64(c.k, at, k_outer), values64(c.v, at, v_outer)
            for p in range(P):
                n = min(int(c.row_lens[r, p]), longest)
                for j in range(h * Hq // c.kv_heads, (h + 1) * Hq // c.kv_heads):
                    see = good.clone()
                    see[max(0, n):] = False
                    if block_ids is not None:
                        ids = block_ids[r, p * lists + j * lists // Hq]
                        see &= torch.isin(torch.arange(longest) // BLOCK, ids.long())
                    if not see.any():
                        continue
                    k, v = K[see], V[see]
                    s = k @ q64[r, p, j] * sm_scale
                    z = torch.logsumexp(s, 0)
                    w = torch.exp(s - z)
                    out[r, p, j], lse[r, p, j] = w @ v, z
                    size = float((k.abs() @ q64[r, p, j].abs()).max() * sm_scale)
                    size_q = float(k.abs().sum(1).max() * q64[r, p, j].abs().max() * sm_scale)
                    e_s = 132 * 2.0 ** -23 * size + 2.0 ** -32 * size_q
                    ltol[r, p, j] = e_s + 2.0 ** -16 + 2.0 ** -22 * abs(float(z))
                    tol[r, p, j] = ((w @ v.abs()) * (2 * (e_s + 2.0 ** -16) + 2.0 ** -11)
                                    + v.abs().sum(0) * 2.0 ** -31 * float(w.max())
                                    + out[r, p, j].abs() * 2.0 ** -8)
    return out, lse, tol, ltol
