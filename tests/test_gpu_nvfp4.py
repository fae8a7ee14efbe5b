"""The NVFP4 key-value cache (needs a GPU): stored bytes bit for bit against the oracle, the
attention against a 64-bit reference, with NaN scales in every place that no row sees."""
import pytest
import torch

import _attn
import _nvfp4
import sparse_attention_indexer_packed_gb300 as idx
from test_gpu_attn import LENS, drafts, draws, lists_for

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def run(c, q, sm_scale=SCALE, block_ids=None, lists=0, lse=True, k_outer=1.0, v_outer=1.0):
    d = _attn.to_device(c)
    R, P, Hq, _ = q.shape
    out = torch.full((R, P, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((R, P, Hq), 7.0, device="cuda") if lse else None
    ws = idx.alloc_attn_workspace(P, Hq, c.kv_heads, lists)
    ws.fill_(0xff)          # no clearing is needed
    head = (q.cuda(), *d.k, *d.v, d.page_table, d.slot_ids, d.row_lens)
    if block_ids is None:
        idx.idx_attn_paged_nvfp4(*head, c.kv_heads, sm_scale, out, l, ws, k_outer, v_outer)
    else:
        idx.idx_attn_blocks_nvfp4(*head, block_ids.cuda(), lists, c.kv_heads, sm_scale, out, l, ws,
                                  k_outer, v_outer)
    return out, l, idx.idx_workspace_errors(ws)


# ---- store ---------------------------------------------------------------------------------
def tokens(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, 3 * H, 128), generator=g)
    x *= torch.exp2(torch.randint(-12, 14, (T, 3 * H, 8, 1), generator=g).float()).expand(-1, -1, -1, 16).reshape(T, 3 * H, 128)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("T,H,values", [(1, 1, False), (1, 2, True), (63, 1, True), (64, 3, True),
                                        (257, 4, True), (1000, 1, False), (5000, 2, True)])
@pytest.mark.parametrize("outers", [(1.0, 1.0), (0.125, 32.0)])
def test_store(T, H, values, outers):
    pages = T // 64 + 4
    src = tokens(T, H, 3 + T)
    src[0, 0] = 0
    src[T // 2, H:, 5] = 4 * src[T // 2, H:, 6]    # ties and zeros of either sign
    src[T // 2, H:, 32:48] = -0.0
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * 64, generator=g)[:T]
    if T > 60:
        slots[5], slots[9], slots[11] = -1, pages * 64, -2 ** 62
    pools = [_nvfp4.plane(pages * H * 64, 5 + i) for i in range(2)]
    dev = [tuple(t.cuda() for t in p) for p in pools]
    d = src.cuda()
    k, v = d[:, H:2 * H], d[:, 2 * H:] if values else None
    idx.idx_store_kv_nvfp4(k, v, slots.cuda(), *dev[0], *(dev[1] if values else (None, None)), H, *outers)
    for i in range(2):
        payload, scale = (t.clone() for t in pools[i])
        if i == 0 or values:
            codes, s = _nvfp4.quantize(src[:, (1 + i) * H:(2 + i) * H], outers[i])
            ok = (slots >= 0) & (slots < pages * 64)
            for h in range(H):
                rows = (slots[ok] // 64 * H + h) * 64 + slots[ok] % 64
                payload[rows], scale[rows] = codes[ok, h], s[ok, h]
        assert torch.equal(dev[i][0].cpu(), payload)
        assert torch.equal(dev[i][1].cpu(), scale)


def test_store_writes_the_index_pools_bytes():
    src = tokens(333, 1, 7)[:, :1].contiguous().cuda()
    slots = torch.randperm(640)[:333].cuda()
    planes = [[t.cuda() for t in _nvfp4.plane(640, 5)] for _ in range(2)]
    idx.idx_store_kv_nvfp4(src, None, slots, *planes[0], None, None, 1)
    idx.idx_store_nvfp4(src[:, 0], slots, tuple(planes[1]))
    for a, b in zip(*planes):
        assert torch.equal(a, b)


def test_store_of_values_that_are_not_finite():
    inf, nan = float("inf"), float("nan")
    src = torch.ones((5, 1, 128), dtype=torch.bfloat16)
    src[0, 0, 3], src[1, 0, 3], src[2, 0, 3] = nan, inf, -inf
    src[3, 0, 3] = -3e38
    src[4, 0, :16] = 2.0 ** -130
    payload, scale = (torch.zeros((64, n), dtype=torch.uint8, device="cuda") for n in (64, 8))
    idx.idx_store_kv_nvfp4(src.cuda(), None, torch.arange(5).cuda(), payload, scale, None, None, 1, 2.0 ** -4)
    x = _nvfp4.values64((payload.cpu(), scale.cpu()), torch.arange(5), 2.0 ** -4)
    assert torch.isnan(x[0, :16]).all() and scale[0, 0] == 0x7f and (payload[0, :8] == 0).all()
    most = 6 * 448 * 2.0 ** -4
    for row, top in ((1, most), (2, -most), (3, -most)):
        assert x[row, 3] == top and (x[row, :3] == 0).all()
    assert (x[4, :16] == 0).all() and scale[4, 0] == 0
    for row in range(5):
        # 1 / outer = 16: scale E4M3(16 / 6) = 2.75, code e2m1(16 / 2.75 = 5.8) = 6
        assert (x[row, 16:] == 6 * 2.75 / 16).all()


# ---- attention -----------------------------------------------------------------------------
# More than 32 packed rows go to the kernel of up to 16 where the page table, which bounds the
# tokens, is narrow, and to the tensor-memory one where it is wide.
TABLES = [None, 60000]


@pytest.mark.parametrize("max_pages", TABLES)
@pytest.mark.parametrize("P,Hq,Hkv", [(1, 1, 1), (1, 16, 2), (1, 4, 4), (2, 6, 2), (4, 16, 1),
                                      (4, 8, 2), (3, 10, 2), (1, 40, 1), (7, 24, 1), (8, 16, 1)])
def test_whole_cache(P, Hq, Hkv, max_pages):
    lens = [drafts(L, P) for L in LENS]
    c = _nvfp4.make(lens, Hkv, 11 + P + Hq, pads=(3, 8), max_pages=max_pages)
    q = draws(len(lens), P, Hq, 5)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


@pytest.mark.parametrize("max_pages", TABLES)
@pytest.mark.parametrize("ctas", [1, 2, 7, 0])
@pytest.mark.parametrize("P,Hq,Hkv", [(1, 8, 2), (4, 16, 1)])
def test_splits_of_a_long_cache(ctas, P, Hq, Hkv, max_pages):
    lens = [drafts(L, P) for L in (5000, 3, 2049, 0, 777)]
    c = _nvfp4.make(lens, Hkv, 21, max_pages=max_pages)
    q = draws(len(lens), P, Hq, 6)
    idx.idx_set_grid_limit(ctas)
    try:
        out, l, flags = run(c, q)
        again, l2, _ = run(c, q)
    finally:
        idx.idx_set_grid_limit(0)
    assert flags == 0
    assert torch.equal(out, again) and torch.equal(l, l2)      # the split's order is fixed
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


@pytest.mark.parametrize("R,P,Hq,Hkv,L", [(40, 1, 16, 8, 200), (300, 1, 8, 2, 40), (170, 2, 8, 1, 300),
                                          (64, 1, 4, 4, 130), (24, 6, 16, 2, 150)])
def test_many_units_dealt_whole(R, P, Hq, Hkv, L):
    g = torch.Generator().manual_seed(R)
    lens = [drafts(int(n), P) for n in torch.randint(max(1, L - 40), L + 1, (R,), generator=g)]
    c = _nvfp4.make(lens, Hkv, 23)
    q = draws(R, P, Hq, 7)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


def test_rows_of_very_different_lengths():
    lens = [[1, 700, 0, 64], [129, 128, 2000, 1]]
    for Hq, max_pages in ((4, None), (8, None), (32, None), (32, 60000), (64, 60000)):
        c = _nvfp4.make(lens, 2, 31, max_pages=max_pages)
        q = draws(2, 4, Hq, 7)
        out, l, flags = run(c, q)
        assert flags == 0
        _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


@pytest.mark.parametrize("more", [0, 200])
@pytest.mark.parametrize("P,Hq,Hkv,lists,topk", [
    (1, 16, 1, 4, 8), (4, 16, 1, 4, 16), (4, 16, 4, 4, 5), (4, 16, 4, 2, 5), (2, 12, 2, 6, 3),
    (16, 4, 1, 4, 4), (5, 40, 1, 2, 6), (1, 1, 1, 1, 256), (17, 2, 1, 2, 3), (8, 16, 1, 1, 4)])
def test_blocks(P, Hq, Hkv, lists, topk, more):
    lens = [drafts(L, P) for L in (0, 1, 64, 129, 1000, 2500, 4097)]
    c = _nvfp4.make(lens, Hkv, 41 + P, pads=(2,), max_pages=4000 if more else None)
    q = draws(len(lens), P, Hq, 8)
    ids = lists_for(lens, lists, topk, 9, P)
    if more:      # longer lists with nothing more in them: the other kernel for many rows
        if topk + more > 256:
            pytest.skip("no list is that long")
        ids = torch.cat([ids, torch.full((*ids.shape[:2], more), -1, dtype=torch.int32)], 2)
    # what a list may hold besides: a block twice, no block, blocks past the row's own
    ids[4, 0, 0] = ids[4, 0, topk // 2]
    ids[5, 1 % (P * lists), -1] = -7
    ids[5, 0, 0] = 40 if topk > 1 else 0
    ids[6, P * lists - 1] = -1
    out, l, flags = run(c, q, block_ids=ids, lists=lists)
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE, ids, lists))


@pytest.mark.parametrize("P,Hq,max_pages", [(1, 8, None), (3, 16, None), (3, 16, 60000)])
@pytest.mark.parametrize("outers", [(1.0, 1.0), (2.0 ** -20, 2.0 ** 30), (2.0 ** 40, 2.0 ** -50)])
def test_outer_scales_and_group_scales_of_every_size(P, Hq, max_pages, outers):
    lens = [drafts(L, P) for L in (900, 65, 1)]
    c = _nvfp4.make(lens, 1, 61, spread=9, max_pages=max_pages)
    q = draws(3, P, Hq, 11)
    out, l, flags = run(c, q, SCALE / outers[0], k_outer=outers[0], v_outer=outers[1])
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE / outers[0], k_outer=outers[0], v_outer=outers[1]))


@pytest.mark.parametrize("Hq,P,max_pages", [(4, 2, None), (16, 4, None), (16, 4, 300000 // 64 * 13), (16, 8, 60000)])
def test_a_token_that_one_draft_row_sees_does_not_reach_the_others(Hq, P, max_pages):
    lens = [[70 + p for p in range(P)]]
    for plane in ("k", "v"):
        c = _nvfp4.make(lens, 1, 71, max_pages=max_pages)
        slot = int(c.slot_ids[0])
        row = int(c.page_table[slot, (70 + P - 2) // 64]) * 64 + (70 + P - 2) % 64   # the last draft's own
        getattr(c, plane)[1][row, 2] = 0x7f
        q = draws(1, P, Hq, 12)
        out, l, _ = run(c, q)
        ref = _nvfp4.reference(c, q, SCALE)
        last = out[0, P - 1].cpu()
        assert torch.isnan(last).any()
        _attn.check(out[:, :P - 1], l[:, :P - 1], tuple(x[:, :P - 1] for x in ref))


def test_bad_pages_are_left_out_and_flagged():
    lens = [[500], [200]]
    for Hq, max_pages in ((4, None), (40, None), (40, 60000)):
        c = _nvfp4.make(lens, 1, 81, max_pages=max_pages)
        slot = int(c.slot_ids[0])
        c.page_table[slot, 2], c.page_table[slot, 5] = c.num_pages, -9
        q = draws(2, 1, Hq, 13)
        out, l, flags = run(c, q)
        assert flags == 1
        _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


def test_long_rows_are_clamped():
    for Hq in (4, 40):
        c = _nvfp4.make([[128], [100]], 1, 83, max_pages=2)
        c.row_lens[0, 0] = 5000
        q = draws(2, 1, Hq, 14)
        out, l, flags = run(c, q)
        assert flags == 4
        c.row_lens[0, 0] = 128
        _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


def test_queries_of_any_size():
    for Hq, max_pages in ((4, None), (40, 60000)):
        c = _nvfp4.make([[300], [65]], 1, 85, max_pages=max_pages)
        q = draws(2, 1, Hq, 15)
        q[0, 0, 0] *= 2.0 ** 100
        q[0, 0, 1] *= 2.0 ** -110
        q[1, 0, 2] = 0
        q[1, 0, 3, ::2] *= 2.0 ** -10
        out, l, flags = run(c, q, 2.0 ** -30)
        assert flags == 0
        ref = _nvfp4.reference(c, q, 2.0 ** -30)
        _attn.check(out, l, ref)


def test_two_captured_calls_and_a_stream_of_their_own():
    P, Hq, Hkv = 2, 8, 1
    c = _nvfp4.make([drafts(L, P) for L in (700, 90)], Hkv, 91)
    d = _attn.to_device(c)
    q = draws(2, P, Hq, 16).cuda()
    out, l = torch.empty_like(q), torch.empty((2, P, Hq), device="cuda")
    ws = idx.alloc_attn_workspace(P, Hq, Hkv)
    call = lambda: idx.idx_attn_paged_nvfp4(q, *d.k, *d.v, d.page_table, d.slot_ids, d.row_lens, Hkv,  # noqa: E731
                                            SCALE, out, l, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (17, 18):
        new = draws(2, P, Hq, seed)
        q.copy_(new)
        graph.replay()
        _attn.check(out, l, _nvfp4.reference(c, new, SCALE))


def test_past_32_bit_offsets():
    rows = 72 << 20                   # 4.8e9 bytes of codes, 6e8 of scales
    pages = rows // 64
    k, v = [(torch.zeros((rows, 64), dtype=torch.uint8, device="cuda"),
             torch.zeros((rows, 8), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    want = [pages - 1, 3, pages // 2 + 1]
    small = _nvfp4.make([[190]], 1, 95, garbage=False)
    small_pages = small.page_table[int(small.slot_ids[0]), :3].tolist()
    for big, p in ((k, small.k), (v, small.v)):
        for a, b in zip(want, small_pages):
            for dst, src in zip(big, p):
                dst[a * 64:a * 64 + 64] = src[b * 64:b * 64 + 64].cuda()
    for Hq, more in ((4, 0), (40, 60000)):
        q = draws(1, 1, Hq, 19)
        out, l = torch.empty_like(q, device="cuda"), torch.empty((1, 1, Hq), device="cuda")
        ws = idx.alloc_attn_workspace(1, Hq, 1)
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        table = i32(want + [-1] * more)
        idx.idx_attn_paged_nvfp4(q.cuda(), *k, *v, table, i32(0), i32([190]), 1, SCALE, out, l, ws)
        assert idx.idx_workspace_errors(ws) == 0
        _attn.check(out, l, _nvfp4.reference(small, q, SCALE))
    src = tokens(2, 1, 20)[:, :1]
    idx.idx_store_kv_nvfp4(src.cuda(), None, torch.tensor([rows - 1, 7]).cuda(), *k, None, None, 1)
    codes, s = _nvfp4.quantize(src)
    assert torch.equal(k[0][[rows - 1, 7]].cpu(), codes[:, 0]) and torch.equal(k[1][[rows - 1, 7]].cpu(), s[:, 0])


def test_a_wait_that_runs_out_is_reported():
    for Hq, max_pages in ((4, None), (40, 60000)):
        c = _nvfp4.make([[900]], 1, 97, max_pages=max_pages)
        q = draws(1, 1, Hq, 21)
        idx.idx_set_wait_limit_ns(20_000_000)
        idx.idx_set_stall_test(1)
        try:
            _, _, flags = run(c, q)
        finally:
            idx.idx_set_stall_test(0)
            idx.idx_set_wait_limit_ns(0)
        assert flags == 2
        out, l, flags = run(c, q)
        assert flags == 0
        _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


def test_no_requests():
    c = _nvfp4.make([[5]], 1, 99)
    d = _attn.to_device(c)
    ws = idx.alloc_attn_workspace(1, 4, 1)
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.empty((0, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
    idx.idx_attn_paged_nvfp4(q, *d.k, *d.v, d.page_table, e(0), e(0, 1), 1, SCALE, q, None, ws)
    assert idx.idx_workspace_errors(ws) == 0
