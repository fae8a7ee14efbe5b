"""Error bounds of one attention row, from the roundings that idx.h states and nothing else.

Scores: 128 exact products summed in fp32 (the tensor cores may truncate, 2^-23 a step) and four
more roundings: e_s = 132 2^-23 max_t sum |q||k| scale.  A query element of the tcgen05 kernel's
e4m3 call is exact within 2^13 of its row's largest and off by 2^-21 of the largest at most.
Weights: e_s, ex2's 2^-22, and the rounding before the product with the values: two bf16, 2^-17;
or one f16, 2^-11 of the weight times value scale, and 2^-28 of the row's largest such product
(f16's subnormals: half of 2^-24, where the largest product is held as 2^3 or more).
Sums: a truncation a product step (two a step of 16 tokens for two bf16) and a factor a piece
that raises the maximum, 2^-22 each.  The result is rounded to bf16 once: 2^-8."""
import torch

import _attn


def reference(c, q, sm_scale, block_ids=None, lists=0, split_query=False, keep=None):
    """out, lse, tol, ltol in float64, as _attn.reference; keep(r, p, j): rows to compute."""
    R, P, Hq, _ = q.shape
    out = torch.zeros((R, P, Hq, _attn.DIM), dtype=torch.float64)
    lse = torch.full((R, P, Hq), -float("inf"), dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(R):
        if not 0 <= int(c.slot_ids[r]) < c.page_table.shape[0]:
            continue
        pages = c.page_table[int(c.slot_ids[r])].tolist()
        for p in range(P):
            n = int(c.row_lens[r, p])
            for j in range(Hq):
                if n <= 0 or (keep is not None and not keep(r, p, j)):
                    continue
                at = _attn.token_rows(pages, n, j * c.kv_heads // Hq, c.kv_heads)
                if block_ids is not None:
                    ids = block_ids[r, p * lists + j * lists // Hq].tolist()
                    at = at[[t for b in sorted({b for b in ids if b >= 0})
                             for t in range(b * _attn.BLOCK, min(n, (b + 1) * _attn.BLOCK))]]
                if not len(at):
                    continue
                k, v = _attn.values64(c.k, at), _attn.values64(c.v, at)
                scale = None if c.dtype == "bf16" else c.v[1][at].double()
                row = q[r, p, j].double()
                s = k @ row * sm_scale
                z = torch.logsumexp(s, 0)
                w = torch.exp(s - z)
                out[r, p, j], lse[r, p, j] = w @ v, z
                tol[r, p, j], ltol[r, p, j] = bounds(row, k, v, scale, w, z, sm_scale, split_query)
    return out, lse, tol, ltol


def bounds(q, k, v, scale, w, z, sm_scale, split_query=False):
    """scale: the value scales of an e4m3 cache, or None."""
    n = len(w)
    e_s = 132 * 2.0 ** -23 * float((k.abs() @ q.abs()).max()) * sm_scale
    if split_query and float(q[q != 0].abs().min()) < 2.0 ** -12 * float(q.abs().max()):
        e_s += 2.0 ** -21 * float(q.abs().max()) * float(k.abs().sum(1).max()) * sm_scale
    steps = (n / 8 + 64) * 2.0 ** -22
    mass = w @ v.abs()
    rounding = 2.0 ** -17 if scale is None else 2.0 ** -11
    tol = mass * (2 * e_s + rounding + 2 * steps) + (w @ v).abs() * 2.0 ** -8
    if scale is not None:
        codes = (v / scale.reshape(-1, 1).clamp_min(2.0 ** -140)).abs()
        tol = tol + 2.0 ** -28 * float((w * scale.flatten()).max()) * codes.sum(0)
    return tol, e_s + steps + 2.0 ** -22 * abs(float(z))


def check(out, lse, ref, rows=None):
    o, l = out.cpu().double(), lse.cpu().double()
    rows = torch.ones_like(l, dtype=torch.bool) if rows is None else rows
    d, dl = (o - ref[0]).abs()[rows], (l - ref[1]).abs()[rows]
    assert torch.isfinite(o[rows]).all() and torch.isfinite(l[rows]).all()
    assert (dl <= ref[3][rows]).all(), float((dl / ref[3][rows]).max())
    assert (d <= ref[2][rows]).all(), float((d / ref[2][rows].clamp_min(1e-300)).max())
