"""Measured cases of the 4-bit key-value cache and of the pass that fills a cache.

Four operators of a sparse-attention decode layer: the store of new keys and values into an
NVFP4 cache, the attention of the newest tokens over such a cache, the attention over the
blocks of it that the index step chose, and the pass from a fused projection to the cache:
norm of the queries and keys head by head, rotation by position (one axis, or several for
images and video), the keys and values stored.

The layouts are the library's: pages of 64 tokens, blocks of 128, head dim 128.  A cache of H
heads is a plane of rows (page * H + head) * 64 + token % 64.  An NVFP4 row is 64 bytes of
e2m1 codes (the even element in the low nibble) and 8 bytes of E4M3 scales, one for each 16
elements: value = code * scale * outer, with one power of two `outer` for the plane.  Draft row
j of a request whose newest length is L sees L - (P - 1) + j tokens.  `own` chooses between the
library's calls and the same operators in elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE, BLOCK, DIM, GROUP = 64, 128, 128, 16
E4M3_MAX, E2M1_MAX = 448.0, 6.0
AMAX_FLOOR = 2.0 ** -96           # smallest amax an fp32 scale is made from
INIT_BLOCKS, LOCAL_BLOCKS = 1, 4  # blocks every list of the index step holds
WORKSPACE_BYTES = 64 << 20        # more than any call below asks for
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token early in a chat: nothing but latency
        {"name": "attn4-1x1k", "op": "attn", "requests": 1, "queries": 1, "q_heads": 16,
         "kv_heads": 2, "context": 1000, "ragged": False},
        # a batch of chats of every age and one graph-padding request, several key heads
        {"name": "attn4-48-ragged", "op": "attn", "requests": 48, "queries": 1, "q_heads": 32,
         "kv_heads": 4, "context": 16384, "ragged": True},
        # long-context decode: what a 4-bit cache is for
        {"name": "attn4-16x131k", "op": "attn", "requests": 16, "queries": 1, "q_heads": 16,
         "kv_heads": 1, "context": 131072, "ragged": False},
        # speculative verify of four draft rows over the whole context (64 rows a key)
        {"name": "attn4-verify-16x131k", "op": "attn", "requests": 16, "queries": 4, "q_heads": 16,
         "kv_heads": 1, "context": 131072, "ragged": False},
        # one request's sparse decode step: 16 blocks a list
        {"name": "blocks4-1x32k", "op": "blocks", "requests": 1, "queries": 1, "q_heads": 16,
         "kv_heads": 1, "lists": 4, "context": 32768, "topk": 16, "ragged": False},
        # the sparse verify step of the 16 x 131K workload: 64 blocks a list
        {"name": "blocks4-verify-16x131k", "op": "blocks", "requests": 16, "queries": 4,
         "q_heads": 16, "kv_heads": 1, "lists": 4, "context": 131072, "topk": 64, "ragged": False},
        # new keys and values of one verify step
        {"name": "store4-64", "op": "store", "tokens": 64, "kv_heads": 2, "values": True},
        # a prefill chunk's keys and values, an odd number of tokens
        {"name": "store4-32001", "op": "store", "tokens": 32001, "kv_heads": 4, "values": True},
        # the projection of one verify step into an e4m3 cache
        {"name": "rope-64", "op": "rope", "tokens": 64, "q_heads": 16, "kv_heads": 2,
         "dtype": "fp8_e4m3", "values": True, "rotary_dim": 128, "interleaved": False, "axes": 1,
         "norm": True, "q_codes": False},
        # that of a prefill chunk into a bf16 cache
        {"name": "rope-16k", "op": "rope", "tokens": 16384, "q_heads": 32, "kv_heads": 4,
         "dtype": "bf16", "values": True, "rotary_dim": 128, "interleaved": False, "axes": 1,
         "norm": True, "q_codes": False},
        # video tokens (time, height, width) into a 4-bit cache, an odd number of them
        {"name": "rope-video-5001", "op": "rope", "tokens": 5001, "q_heads": 16, "kv_heads": 2,
         "dtype": "nvfp4", "values": True, "rotary_dim": 128, "interleaved": False, "axes": 3,
         "norm": True, "q_codes": False},
        # index queries (e4m3, a scale a row) and index keys of a prefill chunk: half of each
        # head rotated, neighbouring elements paired, no values
        {"name": "rope-index-8k", "op": "rope", "tokens": 8192, "q_heads": 4, "kv_heads": 1,
         "dtype": "fp8_e4m3", "values": False, "rotary_dim": 64, "interleaved": True, "axes": 1,
         "norm": True, "q_codes": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(4, 1), (8, 1), (16, 1), (8, 2), (16, 2), (32, 4), (32, 8), (16, 16), (12, 4), (10, 2)]


def draw(rng):
    op = rng.choice(["attn", "attn", "blocks", "blocks", "store", "rope", "rope"])
    if op == "store":
        return {"op": op, "tokens": _log_int(rng, 1, 32001), "kv_heads": rng.choice([1, 2, 4]),
                "values": rng.random() < 0.7}
    q_heads, kv_heads = rng.choice(_HEADS)
    if op == "rope":
        tokens = _log_int(rng, 1, 16384 * 40 // max(40, q_heads + 2 * kv_heads))
        axes = rng.choice([1, 1, 2, 3])
        return {"op": op, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
                "dtype": rng.choice(["bf16", "fp8_e4m3", "nvfp4"]), "values": rng.random() < 0.8,
                "rotary_dim": rng.choice([128, 128, 96, 64, 32]), "interleaved": rng.random() < 0.4,
                "axes": axes, "norm": rng.random() < 0.8, "q_codes": rng.random() < 0.3}
    case = {"op": op, "requests": _log_int(rng, 1, 64), "queries": rng.choice([1, 1, 2, 3, 4, 4]),
            "q_heads": q_heads, "kv_heads": kv_heads, "context": _log_int(rng, 1, 131072),
            "ragged": rng.random() < 0.5}
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


_ROW = {"bf16": 256, "fp8_e4m3": 132, "nvfp4": 72}   # bytes a cached row


def work(case):
    op = case["op"]
    if op == "store":
        planes = 2 if case["values"] else 1
        rows = case["tokens"] * case["kv_heads"] * planes
        return {"bytes": rows * (256 + 72) + 8 * case["tokens"], "flops": 3 * rows * DIM}
    if op == "rope":
        T, Hq, H = case["tokens"], case["q_heads"], case["kv_heads"]
        planes = 2 if case["values"] else 1
        out_q = 132 if case["q_codes"] else 256
        # projection in, queries and cache rows out; a table row, the positions, a slot a token
        nbytes = T * (Hq * (256 + out_q) + planes * H * (256 + _ROW[case["dtype"]])
                      + 4 * case["rotary_dim"] + 4 * case["axes"] + 8)
        return {"bytes": nbytes, "flops": T * ((Hq + H) * 8 + planes * H * 3) * DIM}
    R, P, Hq, Hkv = (case[k] for k in ("requests", "queries", "q_heads", "kv_heads"))
    lens = _lens(case)
    io = R * P * Hq * (DIM * 4 + 4)
    if op == "attn":
        keys = sum(lens) * Hkv
        pairs = sum(max(0, L - (P - 1) + p) for L in lens for p in range(P)) * Hq
    else:
        n_lists = case["lists"]
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
    return {"bytes": keys * 2 * 72 + io, "flops": 4 * pairs * DIM}


# --------------------------------------------------------------------------- formats
def _quantize_rows(x):
    """e4m3 codes and one fp32 scale of each row of x (fp32)."""
    amax = x.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    codes = (x * (E4M3_MAX / amax)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, amax / E4M3_MAX


def _quantize_nvfp4(x):
    """NVFP4 of rows of 128 (fp32, already divided by the outer scale): bytes [.., 64] of two
    codes each and E4M3 scales [.., 8] as bytes.  Half to even, saturating."""
    v = x.reshape(*x.shape[:-1], DIM // GROUP, GROUP)
    scale = (v.abs().amax(-1) / E2M1_MAX).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    a = v.abs() / s
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = torch.where(s > 0, code + 8 * torch.signbit(v).to(torch.uint8), 0).to(torch.uint8)
    code = code.reshape(*x.shape[:-1], DIM // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scale.view(torch.uint8)


def _code_values(payload, dtype):
    """The e2m1 values of packed codes: [.., 64] bytes to [.., 128]."""
    pair = [[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)]
    lut = torch.tensor(pair, dtype=dtype, device=payload.device)
    return lut[payload.int()].flatten(-2)


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _plane(g, rows, dtype, spread=1.0):
    """One plane of a cache that holds N(0, spread) rows: payload, scale."""
    step = 1 << 19
    if dtype == "bf16":
        return torch.randn((rows, DIM), generator=g, device="cuda").to(torch.bfloat16), None
    width, scales, kind = (128, 1, torch.float32) if dtype == "fp8_e4m3" else (64, 8, torch.uint8)
    payload = torch.empty((rows, width), dtype=torch.uint8, device="cuda")
    scale = torch.empty((rows, scales), dtype=kind, device="cuda")
    for a in range(0, rows, step):
        x = torch.randn((min(step, rows - a), DIM), generator=g, device="cuda")
        codes, s = (_quantize_rows if dtype == "fp8_e4m3" else _quantize_nvfp4)(x * spread)
        payload[a:a + step] = codes.view(torch.uint8)
        scale[a:a + step] = s
    return payload, scale


def _slots(g, tokens, pages):
    """Cache slots of new tokens: consecutive in pages of a random order."""
    page = torch.randperm(pages, generator=g, device="cuda")
    t = torch.arange(tokens, device="cuda")
    return page[t // PAGE] * PAGE + t % PAGE


def _pair_axis(case):
    """The axis of each rotated pair: runs of the pairs, the later axes' a little longer."""
    n, axes = case["rotary_dim"] // 2, case["axes"]
    first = n // axes - n // 16 if axes > 1 else n
    return bytes(0 if i < first else 1 + (i - first) * (axes - 1) // (n - first) for i in range(n))


def _positions(case, seed):
    """int32 [axes, T]: text counts on along every axis; the later half is an image sequence
    that moves through height and width and, frame by frame, through time."""
    T, axes = case["tokens"], case["axes"]
    t = np.arange(T, dtype=np.int64)
    start = int(np.random.default_rng(seed).integers(0, 60000))
    pos = np.stack([start + t] * axes)
    if axes > 1:
        half, w = T // 2, 40
        k = t[half:] - half
        frame = (k // (w * 24), k // w % 24, k % w)
        for a in range(axes):
            pos[a, half:] = start + half + frame[3 - axes + a]
    return torch.from_numpy(pos.astype(np.int32)).cuda()


def _rope_table(case, rows=131072):
    """fp32 [rows, rotary_dim]: the cosines of a position's pairs, then the sines."""
    n = case["rotary_dim"] // 2
    freq = 1e6 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    op = case["op"]
    s = {"case": dict(case)}
    H = case["kv_heads"]
    if op in ("store", "rope"):
        T = case["tokens"]
        Hq = case.get("q_heads", 4 * H)
        dtype = case.get("dtype", "nvfp4")
        pages = -(-T // PAGE) + 32
        # the sources are slices of the layer's fused projection: tokens lie apart
        proj = torch.randn((T, Hq + 2 * H, DIM), generator=g, device=dev)
        proj[..., ::31] *= 4          # a few large channels
        proj = proj.to(torch.bfloat16)
        s["q"], s["k"] = proj[:, :Hq], proj[:, Hq:Hq + H]
        s["v"] = proj[:, Hq + H:] if case["values"] else None
        s["k_pool"] = _plane(g, pages * H * PAGE, dtype)
        s["v_pool"] = _plane(g, pages * H * PAGE, dtype) if case["values"] else None
        s["slots"] = _slots(g, T, pages)
        # a layer whose values are small keeps them in units of 2^-4
        s["k_outer"], s["v_outer"] = 1.0, 0.0625 if dtype == "nvfp4" else 1.0
        if op == "store":
            return s
        for name in ("q_weight", "k_weight"):
            w = (1 + 0.1 * torch.randn(DIM, generator=g, device=dev)).to(torch.bfloat16)
            s[name] = w if case["norm"] else None
        s["positions"] = _positions(case, seed)
        s["pair_axis"] = _pair_axis(case)
        s["table"] = _rope_table(case)
        s["out_q"] = torch.empty((T, Hq, DIM), device=dev,
                                 dtype=torch.float8_e4m3fn if case["q_codes"] else torch.bfloat16)
        s["out_q_scale"] = torch.empty((T, Hq), device=dev) if case["q_codes"] else None
        return s
    R, P, Hq = case["requests"], case["queries"], case["q_heads"]
    lens = _lens(case)
    need = [-(-L // PAGE) for L in lens]
    max_pages = max(1, max(need))
    num_pages = sum(need) + 8
    n_slots = R + 3
    s["q"] = (1.5 * torch.randn((R, P, Hq, DIM), generator=g, device=dev)).to(torch.bfloat16)
    s["k_pool"] = _plane(g, num_pages * H * PAGE, "nvfp4")
    s["v_pool"] = _plane(g, num_pages * H * PAGE, "nvfp4", 4.0)
    s["k_outer"], s["v_outer"] = 1.0, 0.25
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
    kp, ks = s["k_pool"]
    vp, vs = s["v_pool"] or (None, None)
    if op == "store":
        idx.idx_store_kv_nvfp4(s["k"], s["v"], s["slots"], kp, ks, vp, vs, case["kv_heads"],
                               s["k_outer"], s["v_outer"])
        return _planes(s)
    if op == "rope":
        idx.idx_norm_rope_store(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], 1e-6,
                                s["table"], s["positions"], s["pair_axis"], case["interleaved"],
                                s["slots"], s["out_q"], s["out_q_scale"], kp, ks, vp, vs,
                                case["dtype"], case["kv_heads"], s["k_outer"], s["v_outer"])
        return _rope_result(s)
    if op == "attn":
        idx.idx_attn_paged_nvfp4(s["q"], kp, ks, vp, vs, s["page_table"], s["slot_ids"],
                                 s["row_lens"], case["kv_heads"], s["sm_scale"], s["out"],
                                 s["out_lse"], s["workspace"], s["k_outer"], s["v_outer"])
    else:
        idx.idx_attn_blocks_nvfp4(s["q"], kp, ks, vp, vs, s["page_table"], s["slot_ids"],
                                  s["row_lens"], s["block_ids"], case["lists"], case["kv_heads"],
                                  s["sm_scale"], s["out"], s["out_lse"], s["workspace"],
                                  s["k_outer"], s["v_outer"])
    return s["out"], s["out_lse"]


def _planes(s):
    """The NVFP4 cache's planes: packed codes, scales as the values they stand for (views)."""
    return [x for pool in (s["k_pool"], s["v_pool"]) if pool is not None
            for x in (pool[0], pool[1].view(torch.float8_e4m3fn))]


def _rows(s):
    """Cache rows of the new tokens' heads, [T, H]."""
    H = s["case"]["kv_heads"]
    slots = s["slots"]
    return ((slots // PAGE)[:, None] * H + torch.arange(H, device=slots.device)) * PAGE + (slots % PAGE)[:, None]


def _rope_result(s):
    """Queries, then the planes as the values they stand for.  Of an NVFP4 plane, where two
    codes share a byte, the new rows' codes are unpacked (e2m1 values are exact in e4m3)."""
    out = [s["out_q"]] + ([s["out_q_scale"]] if s["case"]["q_codes"] else [])
    rows = _rows(s) if s["case"]["dtype"] == "nvfp4" else None
    for pool in (s["k_pool"], s["v_pool"]):
        if pool is None:
            continue
        payload, scale = pool
        if s["case"]["dtype"] == "bf16":
            out.append(payload)
        elif s["case"]["dtype"] == "fp8_e4m3":
            out += [payload.view(torch.float8_e4m3fn), scale]
        else:
            out += [_code_values(payload[rows], torch.float16).to(torch.float8_e4m3fn),
                    scale.view(torch.float8_e4m3fn)]
    return out


def _run_plain(s):
    return {"store": _plain_store, "rope": _plain_rope, "attn": _plain_attn,
            "blocks": _plain_blocks}[s["case"]["op"]](s)


def _put(x, pool, rows, dtype, outer):
    """Rows of fp32 values into a plane."""
    payload, scale = pool
    if dtype == "bf16":
        payload[rows] = x.to(torch.bfloat16)
        return
    codes, sc = _quantize_rows(x) if dtype == "fp8_e4m3" else _quantize_nvfp4(x * (1.0 / outer))
    payload[rows] = codes.view(torch.uint8)
    scale[rows] = sc


def _plain_store(s):
    rows = _rows(s)
    _put(s["k"].float(), s["k_pool"], rows, "nvfp4", s["k_outer"])
    if s["v"] is not None:
        _put(s["v"].float(), s["v_pool"], rows, "nvfp4", s["v_outer"])
    return _planes(s)


def _plain_rope(s):
    case = s["case"]
    n = case["rotary_dim"] // 2
    axis = torch.frombuffer(bytearray(s["pair_axis"]), dtype=torch.uint8).to("cuda", torch.int64)
    pair = torch.arange(n, device="cuda")
    pos = s["positions"].long()[axis].T                               # [T, n]
    cos, sin = s["table"][pos, pair][:, None], s["table"][pos, n + pair][:, None]
    first, second = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, n + pair)

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        a, b = x[..., first], x[..., second]
        y = x.clone()
        y[..., first] = a * cos - b * sin
        y[..., second] = b * cos + a * sin
        return y

    q = turned(s["q"], s["q_weight"])
    if case["q_codes"]:
        codes, scale = _quantize_rows(q)
        s["out_q"].copy_(codes)
        s["out_q_scale"].copy_(scale[..., 0])
    else:
        s["out_q"].copy_(q)
    rows = _rows(s)
    _put(turned(s["k"], s["k_weight"]), s["k_pool"], rows, case["dtype"], s["k_outer"])
    if s["v"] is not None:
        _put(s["v"].float(), s["v_pool"], rows, case["dtype"], s["v_outer"])
    return _rope_result(s)


def _rows_f32(pool, rows, outer):
    """Rows of an NVFP4 plane as fp32 values."""
    payload, scale = pool
    s = scale.view(torch.float8_e4m3fn)[rows].float() * outer
    return _code_values(payload[rows], torch.float32) * s.repeat_interleave(GROUP, -1)


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
    k = _rows_f32(s["k_pool"], rows, s["k_outer"])
    scores = torch.einsum("rphgd,rhtd->rphgt", q, k) * s["sm_scale"]
    v = torch.where(live, _rows_f32(s["v_pool"], rows, s["v_outer"]), 0.0)
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
    k = _rows_f32(s["k_pool"], rows, s["k_outer"])
    scores = torch.einsum("rpugd,rputd->rpugt", q, k) * s["sm_scale"]
    v = torch.where(seen[..., None], _rows_f32(s["v_pool"], rows, s["v_outer"]), 0.0)
    out, lse = _softmax_pv(scores, seen[:, :, :, None], v, "rpugt,rputd->rpugd")
    return out.reshape(R, P, Hq, DIM).to(torch.bfloat16), lse.reshape(R, P, Hq)


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits.  Values are given before their rounding to the
    type they are held in; the 4-bit codes, each a multiple of a scale that is rounded itself,
    have no such value."""
    s = prepare(case, seed)
    return {"store": _exact_store, "rope": _exact_rope, "attn": _exact_attention,
            "blocks": _exact_attention}[case["op"]](case, s)


def _exact_plane(case, x, pool, rows, outer):
    """What a plane's outputs are once the rows [T, H] hold x (64 bits)."""
    payload, scale = pool
    dtype = case.get("dtype", "nvfp4")
    if dtype == "bf16":
        got = payload.double()
        got[rows] = x
        return [got]
    if dtype == "fp8_e4m3":
        got, scales = payload.view(torch.float8_e4m3fn).double(), scale.double()
        top = x.abs().max(2, keepdim=True).values.clamp(min=AMAX_FLOOR)
        got[rows] = x * E4M3_MAX / top
        scales[rows] = top / E4M3_MAX
        return [got, scales]
    scales = scale.view(torch.float8_e4m3fn).double()
    v = x.reshape(*x.shape[:2], DIM // GROUP, GROUP) / outer
    scales[rows] = v.abs().max(3).values / E2M1_MAX
    return [None, scales]


def _exact_rows(case, s):
    H = case["kv_heads"]
    return torch.stack([(s["slots"] // PAGE * H + h) * PAGE + s["slots"] % PAGE for h in range(H)], 1)


def _exact_store(case, s):
    rows = _exact_rows(case, s)
    got = _exact_plane(case, s["k"].double(), s["k_pool"], rows, s["k_outer"])
    if s["v"] is not None:
        got += _exact_plane(case, s["v"].double(), s["v_pool"], rows, s["v_outer"])
    return got


def _exact_rope(case, s):
    n = case["rotary_dim"] // 2
    pos, table = s["positions"].long(), s["table"].double()

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).sum(2, keepdim=True) / DIM + 1e-6).sqrt() * weight.double()
        y = x.clone()
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + n)
            at = pos[s["pair_axis"][i]]
            c, z = table[at, i][:, None], table[at, n + i][:, None]
            y[:, :, a] = x[:, :, a] * c - x[:, :, b] * z
            y[:, :, b] = x[:, :, a] * z + x[:, :, b] * c
        return y

    q = turned(s["q"], s["q_weight"])
    got = [q]
    if case["q_codes"]:
        top = q.abs().max(2, keepdim=True).values.clamp(min=AMAX_FLOOR)
        got = [q * E4M3_MAX / top, (top / E4M3_MAX)[:, :, 0]]
    rows = _exact_rows(case, s)
    got += _exact_plane(case, turned(s["k"], s["k_weight"]), s["k_pool"], rows, s["k_outer"])
    if s["v"] is not None:
        got += _exact_plane(case, s["v"].double(), s["v_pool"], rows, s["v_outer"])
    return got


def _exact_attention(case, s):
    R, P, Hq, H = case["requests"], case["queries"], case["q_heads"], case["kv_heads"]
    out = torch.zeros((R, P, Hq, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((R, P, Hq), -math.inf, dtype=torch.float64, device="cuda")
    slots, lens = s["slot_ids"].tolist(), s["row_lens"].tolist()
    n_lists = case.get("lists", H)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def values(pool, rows, outer):
        payload, scale = pool
        b = payload[rows]
        codes = torch.stack([grid[(b & 15).int()], grid[(b >> 4).int()]], 2).reshape(-1, DIM // GROUP, GROUP)
        held = scale.view(torch.float8_e4m3fn)[rows].double()
        return (codes * held[:, :, None] * outer).reshape(-1, DIM)

    for r in range(R):
        L = max(lens[r])
        if slots[r] < 0 or L <= 0:
            continue
        tok = torch.arange(L, device="cuda")
        page = s["page_table"][slots[r]].long()
        for h in range(H):
            rows = (page[tok // PAGE] * H + h) * PAGE + tok % PAGE
            k, v = values(s["k_pool"], rows, s["k_outer"]), values(s["v_pool"], rows, s["v_outer"])
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
