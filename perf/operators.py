"""Measured cases of the cache-and-attention operators of a sparse-attention decode layer.

Four operators that stand around the index step: the store of new keys and values
into the paged cache, the attention of the newest tokens over the whole cache, the
attention over the 128-token blocks that the index step chose, and the root-mean-square
norm with the residual's addition whose result is held in e4m3 with scales.

The layouts are the library's: pages of 64 tokens, blocks of 128, head dim 128.  A cache
of H heads is a plane of rows (page * H + head) * 64 + token % 64; an e4m3 cache has one
fp32 scale a row beside it.  Draft row j of a request whose newest length is L sees
L - (P - 1) + j tokens.  `own` chooses between the library's calls and the same
operators in elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE, BLOCK, DIM = 64, 128, 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96          # smallest amax a scale is made from
INIT_BLOCKS, LOCAL_BLOCKS = 1, 4  # blocks every list of the index step holds
WORKSPACE_BYTES = 64 << 20       # more than any call below asks for


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token early in a chat: nothing but latency
        {"name": "attn-1x1k", "op": "attn", "dtype": "bf16", "requests": 1, "queries": 1,
         "q_heads": 16, "kv_heads": 2, "context": 1000, "ragged": False},
        # a batch of chats of every age and one graph-padding request, several key heads
        {"name": "attn-48-ragged", "op": "attn", "dtype": "bf16", "requests": 48, "queries": 1,
         "q_heads": 32, "kv_heads": 4, "context": 16384, "ragged": True},
        # long-context decode from an 8-bit cache
        {"name": "attn-16x131k-fp8", "op": "attn", "dtype": "fp8_e4m3", "requests": 16,
         "queries": 1, "q_heads": 16, "kv_heads": 1, "context": 131072, "ragged": False},
        # speculative verify of four draft rows over the whole context (64 rows a key)
        {"name": "attn-verify-16x131k", "op": "attn", "dtype": "bf16", "requests": 16,
         "queries": 4, "q_heads": 16, "kv_heads": 1, "context": 131072, "ragged": False},
        # one request's sparse decode step: 16 blocks a list
        {"name": "blocks-1x32k-fp8", "op": "blocks", "dtype": "fp8_e4m3", "requests": 1,
         "queries": 1, "q_heads": 16, "kv_heads": 1, "lists": 4, "context": 32768, "topk": 16,
         "ragged": False},
        # the sparse verify step of the 16 x 131K workload: 64 blocks a list
        {"name": "blocks-verify-16x131k", "op": "blocks", "dtype": "bf16", "requests": 16,
         "queries": 4, "q_heads": 16, "kv_heads": 1, "lists": 4, "context": 131072, "topk": 64,
         "ragged": False},
        # a mixed batch, some contexts shorter than their list; a list a key head
        {"name": "blocks-24-ragged", "op": "blocks", "dtype": "bf16", "requests": 24, "queries": 2,
         "q_heads": 16, "kv_heads": 2, "lists": 2, "context": 65536, "topk": 32, "ragged": True},
        # new keys and values of one verify step
        {"name": "store-64-fp8", "op": "store", "dtype": "fp8_e4m3", "tokens": 64, "kv_heads": 2,
         "values": True},
        # a prefill chunk's keys and values
        {"name": "store-32k-fp8", "op": "store", "dtype": "fp8_e4m3", "tokens": 32768,
         "kv_heads": 4, "values": True},
        # a prefill chunk's index keys: one head, no values
        {"name": "store-50001-index", "op": "store", "dtype": "bf16", "tokens": 50001,
         "kv_heads": 1, "values": False},
        # the layer's entry at one verify step, scales of 128 elements
        {"name": "norm-64x6144", "op": "norm", "tokens": 64, "dim": 6144, "group": 128},
        # and over a prefill chunk, one scale a row
        {"name": "norm-16000x5120", "op": "norm", "tokens": 16000, "dim": 5120, "group": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(4, 1), (8, 1), (16, 1), (8, 2), (16, 2), (32, 4), (32, 8), (16, 16), (12, 4), (10, 2)]
_LISTED_BYTES = 16 * 131072 * 2 * DIM * 2    # the largest listed case reads this much


def draw(rng):
    op = rng.choice(["attn", "attn", "blocks", "blocks", "store", "norm"])
    if op == "norm":
        dim = rng.choice([128, 1024, 2048, 3000, 4096, 5120, 6144, 7168, 8192, 12288, 1001])
        tokens = _log_int(rng, 1, 16000 * 5120 // max(dim, 5120))
        return {"op": op, "tokens": tokens, "dim": dim, "group": rng.choice([0, 128])}
    dtype = rng.choice(["bf16", "fp8_e4m3"])
    if op == "store":
        return {"op": op, "dtype": dtype, "tokens": _log_int(rng, 1, 32768),
                "kv_heads": rng.choice([1, 2, 4]), "values": rng.random() < 0.7}
    q_heads, kv_heads = rng.choice(_HEADS)
    case = {"op": op, "dtype": dtype, "requests": _log_int(rng, 1, 64),
            "queries": rng.choice([1, 1, 2, 3, 4, 4]), "q_heads": q_heads, "kv_heads": kv_heads,
            "context": _log_int(rng, 1, 131072), "ragged": rng.random() < 0.5}
    if op == "blocks":
        case["lists"] = rng.choice([n for n in (1, 2, 4, 8) if q_heads % n == 0
                                    and (n % kv_heads == 0 or kv_heads % n == 0)])
        case["topk"] = _log_int(rng, 8, 64)
        units = max(case["lists"], kv_heads)
        while case["requests"] * case["queries"] * units * min(
                case["topk"] * BLOCK, case["context"]) > 16 * 4 * 4 * 64 * BLOCK:
            case["requests"] = max(1, case["requests"] // 2)
            case["topk"] = max(8, case["topk"] * 2 // 3)
    # no more cache than the largest listed case, and no more products
    while (case["requests"] * case["context"] * kv_heads > 16 * 131072
           or case["requests"] * case["context"] * case["queries"] * q_heads > 16 * 131072 * 64):
        case["context"] = max(1, case["context"] // 2)
    return case


def _lens(case):
    """Newest length of each request (0: a graph-padding request), from the case alone."""
    rng = random.Random("%(requests)d/%(context)d/%(ragged)s" % case)
    n, ctx = case["requests"], case["context"]
    if not case["ragged"]:
        return [rng.randint(max(1, ctx * 7 // 8), ctx) for _ in range(n)]
    lens = [_log_int(rng, 1, ctx) for _ in range(n)]
    if n >= 8:
        lens[n // 2] = 0
    return lens


def _block_lists(case, seed):
    """[R, P, lists, topk] block ids as the index step gives them: the forced blocks, then
    chosen ones, then -1; a draft row differs from the one before in an eighth of its list."""
    R, P, n_lists, topk = case["requests"], case["queries"], case["lists"], case["topk"]
    g = np.random.default_rng(seed)
    ids = np.full((R, P, n_lists, topk), -1, np.int32)
    for r, L in enumerate(_lens(case)):
        for li in range(n_lists):
            nb = -(-L // BLOCK)
            pool = g.permutation(nb)
            pool = pool[(pool >= INIT_BLOCKS) & (pool < nb - LOCAL_BLOCKS)]
            c = max(0, min(topk - INIT_BLOCKS - LOCAL_BLOCKS, len(pool)))
            chosen, spare = pool[:c].copy(), pool[c:]
            used = 0
            for p in range(P):
                if p and c:
                    k = min(max(1, c // 8), len(spare) - used)
                    chosen[g.permutation(c)[:k]] = spare[used:used + k]
                    used += k
                nbp = max(0, -(-(L - (P - 1) + p) // BLOCK))
                forced = sorted(set(range(min(INIT_BLOCKS, nbp))) | set(range(max(0, nbp - LOCAL_BLOCKS), nbp)))
                row = forced + [b for b in chosen.tolist() if b < nbp and b not in forced]
                ids[r, p, li, :min(topk, len(row))] = row[:topk]
    return ids


def work(case):
    op = case["op"]
    if op == "norm":
        T, n = case["tokens"], case["dim"]
        groups = -(-n // case["group"]) if case["group"] else 1
        # x, residual in; residual, codes, scales out; the weight once
        return {"bytes": T * n * 7 + T * groups * 4 + 2 * n, "flops": 6 * T * n}
    row = 256 if case["dtype"] == "bf16" else 132
    if op == "store":
        planes = 2 if case["values"] else 1
        rows = case["tokens"] * case["kv_heads"] * planes
        return {"bytes": rows * (256 + row) + 8 * case["tokens"], "flops": 3 * rows * DIM}
    R, P, Hq, Hkv = (case[k] for k in ("requests", "queries", "q_heads", "kv_heads"))
    lens = _lens(case)
    io = R * P * Hq * (DIM * 4 + 4)
    if op == "attn":
        keys = sum(lens) * Hkv
        pairs = sum(max(0, L - (P - 1) + p) for L in lens for p in range(P)) * Hq
    else:
        n_lists = case["lists"]
        units = max(n_lists, Hkv)
        keys = pairs = 0
        ids = _block_lists(case, 0)
        for r, L in enumerate(lens):
            for h in range(Hkv):
                # the lists that this key head's query heads go by
                own_lists = range(h * n_lists // Hkv, max(h * n_lists // Hkv + 1, (h + 1) * n_lists // Hkv))
                seen = ids[r][:, list(own_lists)]
                blocks = set(seen[seen >= 0].tolist())
                keys += sum(min(BLOCK, L - b * BLOCK) for b in blocks)
            for p in range(P):
                Lp = L - (P - 1) + p
                b = ids[r, p][ids[r, p] >= 0]
                pairs += int(np.minimum(BLOCK, np.maximum(0, Lp - b.astype(np.int64) * BLOCK)).sum()) * (Hq // n_lists)
        io += ids.size * 4
    return {"bytes": keys * 2 * row + io, "flops": 4 * pairs * DIM}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantize(x):
    """e4m3 codes and fp32 scales of the rows of x (fp32)."""
    amax = x.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    codes = (x * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, amax / E4M3_MAX


def _plane(g, rows, dtype):
    """One plane of a cache that holds N(0,1) rows: payload, scale."""
    step = 1 << 21
    if dtype == "bf16":
        payload = torch.empty((rows, DIM), dtype=torch.bfloat16, device="cuda")
        for a in range(0, rows, step):
            payload[a:a + step].normal_(generator=g)
        return payload, None
    payload = torch.empty((rows, DIM), dtype=torch.uint8, device="cuda")
    scale = torch.empty((rows, 1), dtype=torch.float32, device="cuda")
    for a in range(0, rows, step):
        x = torch.randn((min(step, rows - a), DIM), generator=g, device="cuda")
        codes, s = _quantize(x)
        payload[a:a + step] = codes.view(torch.uint8)
        scale[a:a + step] = s
    return payload, scale


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    op = case["op"]
    s = {"case": dict(case)}
    if op == "norm":
        T, n = case["tokens"], case["dim"]
        s["x"] = torch.randn((T, n), generator=g, device=dev).to(torch.bfloat16)
        # a residual stream: larger than what a layer adds, with a few large channels
        res = torch.randn((T, n), generator=g, device=dev) * 4
        res[:, ::97] *= 8
        s["residual"] = res.to(torch.bfloat16)
        s["weight"] = (1 + 0.1 * torch.randn(n, generator=g, device=dev)).to(torch.bfloat16)
        s["out"] = torch.empty((T, n), dtype=torch.float8_e4m3fn, device=dev)
        s["out_scale"] = torch.empty((T, -(-n // case["group"]) if case["group"] else 1), device=dev)
        s["out_residual"] = torch.empty((T, n), dtype=torch.bfloat16, device=dev)
        return s
    H = case["kv_heads"]
    if op == "store":
        T = case["tokens"]
        pages = -(-T // PAGE) + 32
        planes = 2 if case["values"] else 1
        # the source is a slice of the layer's fused projection: tokens lie apart
        proj = torch.randn((T, (4 + planes) * H, DIM), generator=g, device=dev).to(torch.bfloat16)
        s["k"] = proj[:, 4 * H:5 * H]
        s["v"] = proj[:, 5 * H:6 * H] if case["values"] else None
        s["k_pool"] = _plane(g, pages * H * PAGE, case["dtype"])
        s["v_pool"] = _plane(g, pages * H * PAGE, case["dtype"]) if case["values"] else None
        page = torch.randperm(pages, generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["slots"] = page[t // PAGE] * PAGE + t % PAGE
        return s
    R, P, Hq = case["requests"], case["queries"], case["q_heads"]
    lens = _lens(case)
    need = [-(-L // PAGE) for L in lens]
    max_pages = max(1, max(need))
    num_pages = sum(need) + 8
    n_slots = R + 3
    s["q"] = (1.5 * torch.randn((R, P, Hq, DIM), generator=g, device=dev)).to(torch.bfloat16)
    s["k_pool"] = _plane(g, num_pages * H * PAGE, case["dtype"])
    s["v_pool"] = _plane(g, num_pages * H * PAGE, case["dtype"])
    order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    slots = torch.randperm(n_slots, generator=g, device=dev)[:R].to(torch.int32).tolist()
    table = torch.zeros((n_slots, max_pages), dtype=torch.int32, device=dev)
    at = 0
    for r in range(R):
        table[slots[r], :need[r]] = order[at:at + need[r]]
        at += need[r]
        if lens[r] == 0:
            slots[r] = -1
    s["page_table"] = table
    s["slot_ids"] = torch.tensor(slots, dtype=torch.int32, device=dev)
    s["row_lens"] = torch.tensor([[max(0, L - (P - 1) + p) for p in range(P)] for L in lens],
                                 dtype=torch.int32, device=dev)
    s["sm_scale"] = DIM ** -0.5
    s["out"] = torch.empty((R, P, Hq, DIM), dtype=torch.bfloat16, device=dev)
    s["out_lse"] = torch.empty((R, P, Hq), device=dev)
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    if op == "blocks":
        s["block_ids"] = torch.from_numpy(_block_lists(case, seed)).to(dev).reshape(
            R, P * case["lists"], case["topk"])
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_attention_indexer_packed_gb300 as idx
    case = s["case"]
    op = case["op"]
    if op == "norm":
        idx.idx_add_rmsnorm_fp8(s["x"], s["residual"], s["weight"], 1e-6, case["group"], s["out"],
                                s["out_scale"], s["out_residual"])
        return s["out"], s["out_scale"], s["out_residual"]
    kp, ks = s["k_pool"]
    if op == "store":
        vp, vs = s["v_pool"] or (None, None)
        idx.idx_store_kv(s["k"], s["v"], s["slots"], kp, ks, vp, vs, case["dtype"], case["kv_heads"])
        return _pools(s)
    vp, vs = s["v_pool"]
    if op == "attn":
        idx.idx_attn_paged(s["q"], kp, ks, vp, vs, case["dtype"], s["page_table"], s["slot_ids"],
                           s["row_lens"], case["kv_heads"], s["sm_scale"], s["out"], s["out_lse"],
                           s["workspace"])
    else:
        idx.idx_attn_blocks(s["q"], kp, ks, vp, vs, case["dtype"], s["page_table"], s["slot_ids"],
                            s["row_lens"], s["block_ids"], case["lists"], case["kv_heads"],
                            s["sm_scale"], s["out"], s["out_lse"], s["workspace"])
    return s["out"], s["out_lse"]


def _pools(s):
    """The cache's planes as the values they stand for (views, nothing is copied)."""
    out = []
    for pool in (s["k_pool"], s["v_pool"]):
        if pool is not None:
            payload, scale = pool
            out.append(payload if scale is None else payload.view(torch.float8_e4m3fn))
            if scale is not None:
                out.append(scale)
    return out


def _run_plain(s):
    return {"norm": _plain_norm, "store": _plain_store, "attn": _plain_attn,
            "blocks": _plain_blocks}[s["case"]["op"]](s)


def _plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    T, n = x.shape
    h = x + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w
    group = s["case"]["group"] or n
    pad = -n % group
    if pad:
        y = torch.nn.functional.pad(y, (0, pad))
    codes, scale = _quantize(y.reshape(T, -1, group))
    return codes.reshape(T, -1)[:, :n].contiguous(), scale.reshape(T, -1), h.to(torch.bfloat16)


def _store_plane(src, pool, rows):
    payload, scale = pool
    if scale is None:
        payload[rows] = src
    else:
        codes, sc = _quantize(src.float())
        payload[rows] = codes.view(torch.uint8)
        scale[rows] = sc


def _plain_store(s):
    H = s["case"]["kv_heads"]
    slots = s["slots"]
    rows = ((slots // PAGE)[:, None] * H + torch.arange(H, device=slots.device)) * PAGE + (slots % PAGE)[:, None]
    _store_plane(s["k"], s["k_pool"], rows)
    if s["v"] is not None:
        _store_plane(s["v"], s["v_pool"], rows)
    return _pools(s)


def _rows_f32(pool, rows):
    """The cache rows as fp32 values."""
    payload, scale = pool
    if scale is None:
        return payload[rows].float()
    return payload[rows].view(torch.float8_e4m3fn).float() * scale[rows]


def _softmax_pv(scores, seen, v, dims):
    """Masked softmax over the last axis, times v by the einsum `dims`: out and lse."""
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum(dims, p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (torch.log(total) + top)[..., 0]


def _plain_attn(s):
    case = s["case"]
    R, P, Hq, H = case["requests"], case["queries"], case["q_heads"], case["kv_heads"]
    table, slots = s["page_table"], s["slot_ids"].long()
    lens = torch.where((slots >= 0)[:, None], s["row_lens"], 0)
    pages = table[slots.clamp_min(0)].long()                                    # [R, pages]
    n = pages.shape[1] * PAGE
    t = torch.arange(n, device="cuda")
    heads = torch.arange(H, device="cuda")
    rows = (pages[:, t // PAGE][:, None] * H + heads[:, None]) * PAGE + t % PAGE  # [R, H, n]
    live = (t < lens.amax(1)[:, None])[:, None, :, None]
    q = s["q"].float().reshape(R, P, H, Hq // H, DIM)
    scores = torch.einsum("rphgd,rhtd->rphgt", q, _rows_f32(s["k_pool"], rows)) * s["sm_scale"]
    v = torch.where(live, _rows_f32(s["v_pool"], rows), 0.0)
    seen = (t < lens[..., None])[:, :, None, None]
    out, lse = _softmax_pv(scores, seen, v, "rphgt,rhtd->rphgd")
    return out.reshape(R, P, Hq, DIM).to(torch.bfloat16), lse.reshape(R, P, Hq)


def _plain_blocks(s):
    case = s["case"]
    R, P, Hq, H, n_lists = (case[k] for k in ("requests", "queries", "q_heads", "kv_heads", "lists"))
    units = max(H, n_lists)        # query heads of one list and one key head
    u = torch.arange(units, device="cuda")
    slots = s["slot_ids"].long()
    lens = torch.where((slots >= 0)[:, None], s["row_lens"], 0)
    ids = s["block_ids"].reshape(R, P, n_lists, -1)[:, :, u * n_lists // units].long()
    t = (ids[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(R, P, units, -1)
    seen = (t >= 0) & (t < lens[:, :, None, None])
    t = torch.where(seen, t, 0)
    page = s["page_table"].long()[slots.clamp_min(0)[:, None, None, None], t // PAGE]
    rows = (page * H + (u * H // units)[:, None]) * PAGE + t % PAGE               # [R, P, U, n]
    q = s["q"].float().reshape(R, P, units, Hq // units, DIM)
    scores = torch.einsum("rpugd,rputd->rpugt", q, _rows_f32(s["k_pool"], rows)) * s["sm_scale"]
    v = torch.where(seen[..., None], _rows_f32(s["v_pool"], rows), 0.0)
    out, lse = _softmax_pv(scores, seen[:, :, :, None], v, "rpugt,rputd->rpugd")
    return out.reshape(R, P, Hq, DIM).to(torch.bfloat16), lse.reshape(R, P, Hq)


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits.  Codes are given before their rounding to
    8 bits: the quotient of the value and its group's scale."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "store": _exact_store, "attn": _exact_attention,
            "blocks": _exact_attention}[case["op"]](case, s)


def _exact_norm(case, s):
    n, group = case["dim"], case["group"] or case["dim"]
    h = s["x"].double() + s["residual"].double()
    out = torch.empty_like(h)
    scales = []
    rms = ((h * h).sum(1) / n + 1e-6).sqrt()
    for a in range(0, n, group):
        y = h[:, a:a + group] / rms[:, None] * s["weight"][a:a + group].double()
        scale = torch.maximum(y.abs().max(1).values, torch.tensor(AMAX_FLOOR, dtype=torch.float64, device="cuda")) / E4M3_MAX
        out[:, a:a + group] = y / scale[:, None]
        scales.append(scale)
    return out, torch.stack(scales, 1), h


def _exact_store(case, s):
    H = case["kv_heads"]
    got = []
    for src, pool in ((s["k"], s["k_pool"]), (s["v"], s["v_pool"])):
        if pool is None:
            continue
        payload, scale = pool
        if scale is None:
            plane = payload.double()
        else:
            plane, scales = payload.view(torch.float8_e4m3fn).double(), scale.double()
        for h in range(H):
            at = (s["slots"] // PAGE * H + h) * PAGE + s["slots"] % PAGE
            x = src[:, h].double()
            if scale is not None:
                top = x.abs().max(1, keepdim=True).values.clamp(min=AMAX_FLOOR)
                scales[at] = top / E4M3_MAX
                x = x * E4M3_MAX / top
            plane[at] = x
        got.append(plane)
        if scale is not None:
            got.append(scales)
    return got


def _exact_attention(case, s):
    R, P, Hq, H = case["requests"], case["queries"], case["q_heads"], case["kv_heads"]
    out = torch.zeros((R, P, Hq, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((R, P, Hq), -math.inf, dtype=torch.float64, device="cuda")
    slots, lens = s["slot_ids"].tolist(), s["row_lens"].tolist()
    n_lists = case.get("lists", H)

    def values(pool, rows):
        payload, scale = pool
        if scale is None:
            return payload[rows].double()
        return payload[rows].view(torch.float8_e4m3fn).double() * scale[rows].double()

    for r in range(R):
        L = max(lens[r])
        if slots[r] < 0 or L <= 0:
            continue
        tok = torch.arange(L, device="cuda")
        page = s["page_table"][slots[r]].long()
        for h in range(H):
            rows = (page[tok // PAGE] * H + h) * PAGE + tok % PAGE
            k, v = values(s["k_pool"], rows), values(s["v_pool"], rows)
            for p in range(P):
                if lens[r][p] <= 0:
                    continue
                for head0 in range(h * Hq // H, (h + 1) * Hq // H, Hq // max(H, n_lists)):
                    heads = slice(head0, head0 + Hq // max(H, n_lists))
                    if case["op"] == "blocks":
                        ids = s["block_ids"][r, p * n_lists + head0 * n_lists // Hq].long()
                        at = (ids[ids >= 0, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten()
                        at = at[at < lens[r][p]]
                    else:
                        at = slice(0, lens[r][p])
                    x = s["q"][r, p, heads].double() @ k[at].T * s["sm_scale"]
                    z = torch.logsumexp(x, 1)
                    lse[r, p, heads] = z
                    out[r, p, heads] = torch.exp(x - z[:, None]) @ v[at]
    return out, lse
