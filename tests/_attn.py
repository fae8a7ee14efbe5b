"""Seeded caches and a 64-bit reference for the attention tests (plain loops over rows)."""
import dataclasses
import math

import torch

PAGE, BLOCK, DIM = 64, 128, 128


@dataclasses.dataclass
class Cache:
    dtype: str
    kv_heads: int
    num_pages: int
    k: tuple            # (payload, scale) on the device
    v: tuple
    page_table: torch.Tensor
    slot_ids: torch.Tensor
    row_lens: torch.Tensor

    def args(self):
        return (*self.k, *self.v, self.dtype, self.page_table, self.slot_ids, self.row_lens)


def quantize(x):
    amax = x.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -96)
    codes = (x * (448.0 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), amax / 448.0


def plane(rows, dtype, seed, spread=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, DIM), generator=g)
    if spread:   # value scales that differ by many powers of two
        x *= torch.exp2(torch.randint(-12, 13, (rows, 1), generator=g).float())
    if dtype == "bf16":
        return x.to(torch.bfloat16), None
    return quantize(x)


def values64(p, rows):
    payload, scale = p
    if scale is None:
        return payload[rows].double()
    return payload[rows].view(torch.float8_e4m3fn).float().double() * scale[rows].double()


def make(dtype, lens, kv_heads, seed, pads=(), garbage=True, max_pages=None, spread=False):
    """lens: [R][P].  Everything the rows do not see is NaN when garbage is set."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    need = [0 if r in pads else -(-max(0, max(lens[r])) // PAGE) for r in range(R)]
    max_pages = max_pages or max(1, max(need)) + 1
    num_pages = sum(need) + 5
    order = torch.randperm(num_pages, generator=g).tolist()
    table = torch.full((R + 4, max_pages), -1 if garbage else 0, dtype=torch.int32)
    slots = torch.randperm(R + 4, generator=g)[:R].to(torch.int32)
    rows = num_pages * kv_heads * PAGE
    k, v = plane(rows, dtype, seed + 1), plane(rows, dtype, seed + 2, spread)
    seen = torch.zeros(rows, dtype=torch.bool)
    for r in range(R):
        if r in pads:
            slots[r] = -1 if r % 2 else R + 4
            continue
        pages = [order.pop() for _ in range(need[r])]
        table[int(slots[r]), :need[r]] = torch.tensor(pages, dtype=torch.int32)
        for h in range(kv_heads):
            seen[token_rows(pages, max(0, max(lens[r])), h, kv_heads)] = True
    if garbage:
        for payload, scale in (k, v):
            if scale is None:
                payload[~seen] = float("nan")
            else:
                payload[~seen] = 0x7f
                scale[~seen] = float("nan")
    return Cache(dtype, kv_heads, num_pages, k, v, table, slots,
                 torch.tensor(lens, dtype=torch.int32))


def to_device(c, dev="cuda"):
    move = lambda p: tuple(None if t is None else t.to(dev) for t in p)  # noqa: E731
    return dataclasses.replace(c, k=move(c.k), v=move(c.v), page_table=c.page_table.to(dev),
                               slot_ids=c.slot_ids.to(dev), row_lens=c.row_lens.to(dev))


def token_rows(pages, n, h, kv_heads):
    t = torch.arange(n)
    return (torch.tensor(pages, dtype=torch.int64)[t // PAGE] * kv_heads + h) * PAGE + t % PAGE if n else t


def reference(c, q, sm_scale, block_ids=None, lists=0):
    """out, lse in float64 and, per output, the bound on the error that the kernel's roundings
    allow (see tolerances())."""
    R, P, Hq, _ = q.shape
    out = torch.zeros((R, P, Hq, DIM), dtype=torch.float64)
    lse = torch.full((R, P, Hq), -math.inf, dtype=torch.float64)
    tol = torch.zeros((R, P, Hq, DIM), dtype=torch.float64)
    ltol = torch.zeros((R, P, Hq), dtype=torch.float64)
    q64 = q.double()
    for r in range(R):
        slot = int(c.slot_ids[r])
        if not 0 <= slot < c.page_table.shape[0]:
            continue
        pages = c.page_table[slot].tolist()
        for p in range(P):
            n = min(int(c.row_lens[r, p]), c.page_table.shape[1] * PAGE)
            if n <= 0:
                continue
            for j in range(Hq):
                h = j * c.kv_heads // Hq
                at = token_rows(pages, n, h, c.kv_heads)
                if block_ids is not None:
                    ids = block_ids[r, p * lists + j * lists // Hq].tolist()
                    keep = [i for b in sorted({b for b in ids if b >= 0})
                            for i in range(b * BLOCK, min(n, b * BLOCK + BLOCK))]
                    at = at[torch.tensor(keep, dtype=torch.int64)]
                good = (at // (PAGE * c.kv_heads) >= 0) & (at // (PAGE * c.kv_heads) < c.num_pages)
                at = at[good]
                if not len(at):
                    continue
                k, v = values64(c.k, at), values64(c.v, at)
                s = k @ q64[r, p, j] * sm_scale
                z = torch.logsumexp(s, 0)
                w = torch.exp(s - z)
                out[r, p, j] = w @ v
                lse[r, p, j] = z
                size = float((k.abs() @ q64[r, p, j].abs()).max() * sm_scale)
                tol[r, p, j], ltol[r, p, j] = tolerances(c, at, w, v, out[r, p, j], z, size)
    return out, lse, tol, ltol


def tolerances(c, at, w, v, out, z, size):
    """Error bounds of one row.
    Scores: 128 products summed in fp32 (the tensor cores may truncate: 2^-23 a step) and two
    more roundings: e_s = (128 + 4) 2^-23 size, size = max_t sum |q||k| scale.
    lse: e_s, ex2's 2^-22, and a sum whose terms go through at most 64 roundings a level.
    out: each weight is off by e_s + 2^-9 (bf16) or 2^-11 and 2^-25 of the largest value scale
    (f16, its subnormals), against sum w |v|; then one bf16 rounding of the result."""
    e_s = 132 * 2.0 ** -23 * size
    ltol = e_s + 2.0 ** -16 + 2.0 ** -22 * abs(float(z))
    mass = w @ v.abs()
    step = 2.0 ** -9 if c.dtype == "bf16" else 2.0 ** -11
    tol = mass * (2 * (e_s + 2.0 ** -16) + step) + out.abs() * 2.0 ** -8
    if c.dtype != "bf16":
        # 2^-25 absolute, in units of the largest scale (rounded up to a power of two), times the code
        tol = tol + len(at) * 2.0 ** -25 * 2 * float(c.v[1][at].max()) * 448 * float(w.max())
    return tol, ltol


def check(got_out, got_lse, ref):
    out, lse, tol, ltol = ref
    o, l = got_out.cpu().double(), got_lse.cpu().double()
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(l), empty)
    assert torch.equal(o[empty], torch.zeros_like(o[empty]))
    d = (l - lse).abs()[~empty]
    assert (d <= ltol[~empty]).all(), float((d / ltol[~empty]).max())
    d = (o - out).abs()
    assert torch.isfinite(o).all()
    assert (d <= tol).all(), float((d / tol.clamp_min(1e-300)).max())
