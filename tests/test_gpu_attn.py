"""idx_attn_paged / idx_attn_blocks against a 64-bit reference (needs a GPU): shapes, lengths
and masks where a split, packed, paged kernel can go wrong, with NaN in every place of the
cache that no row sees."""
import pytest
import torch

import _attn
import sparse_attention_indexer_packed_gb300 as idx

pytestmark = pytest.mark.gpu
DTYPES = ["bf16", "fp8_e4m3"]


def draws(R, P, Hq, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((R, P, Hq, 128), generator=g)).to(torch.bfloat16)


def run(c, q, sm_scale=128 ** -0.5, block_ids=None, lists=0, lse=True, ws=None):
    d = _attn.to_device(c)
    R, P, Hq, _ = q.shape
    out = torch.full((R, P, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((R, P, Hq), 7.0, device="cuda") if lse else None
    if ws is None:
        ws = idx.alloc_attn_workspace(P, Hq, c.kv_heads, lists)
        ws.fill_(0xff)      # no clearing is needed
    if block_ids is None:
        idx.idx_attn_paged(q.cuda(), *d.args(), c.kv_heads, sm_scale, out, l, ws)
    else:
        idx.idx_attn_blocks(q.cuda(), *d.args(), block_ids.cuda(), lists, c.kv_heads, sm_scale, out, l, ws)
    flags = idx.idx_workspace_errors(ws)
    return out, l, flags


def drafts(L, P):
    return [max(0, L - (P - 1) + p) for p in range(P)]


LENS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 1000]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P,Hq,Hkv", [(1, 1, 1), (1, 16, 2), (1, 4, 4), (2, 6, 2), (4, 16, 1),
                                      (4, 8, 2), (3, 10, 2), (1, 40, 1), (7, 24, 1), (8, 16, 1)])
def test_whole_cache(dtype, P, Hq, Hkv):
    lens = [drafts(L, P) for L in LENS]
    c = _attn.make(dtype, lens, Hkv, 11 + P + Hq, pads=(3, 8))
    q = draws(len(lens), P, Hq, 5)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ctas", [1, 2, 7, 0])
@pytest.mark.parametrize("P,Hq,Hkv", [(1, 8, 2), (4, 16, 1)])
def test_splits_of_a_long_cache(dtype, ctas, P, Hq, Hkv):
    lens = [drafts(L, P) for L in (5000, 3, 2049, 0, 777)]
    c = _attn.make(dtype, lens, Hkv, 21)
    q = draws(len(lens), P, Hq, 6)
    idx.idx_set_grid_limit(ctas)
    try:
        out, l, flags = run(c, q)
        again, l2, _ = run(c, q)
    finally:
        idx.idx_set_grid_limit(0)
    assert flags == 0
    assert torch.equal(out, again) and torch.equal(l, l2)      # the split's order is fixed
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


def test_rows_of_very_different_lengths():
    lens = [[1, 700, 0, 64], [129, 128, 2000, 1]]
    for dtype in DTYPES:
        c = _attn.make(dtype, lens, 2, 31)
        q = draws(2, 4, 8, 7)
        out, l, flags = run(c, q)
        assert flags == 0
        _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


def lists_for(lens, n_lists, topk, seed, P):
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    ids = torch.full((R, P * n_lists, topk), -1, dtype=torch.int32)
    for r in range(R):
        for p in range(P):
            nb = -(-max(lens[r]) // 128)
            for li in range(n_lists):
                pick = torch.randperm(max(1, nb), generator=g)[:topk].to(torch.int32)
                ids[r, p * n_lists + li, :len(pick)] = pick
    return ids


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P,Hq,Hkv,lists,topk", [
    (1, 16, 1, 4, 8), (4, 16, 1, 4, 16), (4, 16, 4, 4, 5), (4, 16, 4, 2, 5), (2, 12, 2, 6, 3),
    (16, 4, 1, 4, 4), (5, 40, 1, 2, 6), (1, 1, 1, 1, 256), (17, 2, 1, 2, 3), (8, 16, 1, 1, 4)])
def test_blocks(dtype, P, Hq, Hkv, lists, topk):
    lens = [drafts(L, P) for L in (0, 1, 64, 129, 1000, 2500, 4097)]
    c = _attn.make(dtype, lens, Hkv, 41 + P, pads=(2,))
    q = draws(len(lens), P, Hq, 8)
    ids = lists_for(lens, lists, topk, 9, P)
    # what a list may hold besides: a block twice, no block, blocks past the row's own
    ids[4, 0, 0] = ids[4, 0, topk // 2]
    ids[5, 1 % (P * lists), -1] = -7
    ids[5, 0, 0] = 40 if topk > 1 else 0
    ids[6, P * lists - 1] = -1
    out, l, flags = run(c, q, block_ids=ids, lists=lists)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5, ids, lists))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ids_of_any_value_are_left_out(dtype):
    lens = [[300], [128]]
    c = _attn.make(dtype, lens, 1, 51)
    q = draws(2, 1, 4, 10)
    ids = torch.tensor([[[2 ** 31 - 1, -2 ** 31, 2, 3, 0, 2 ** 24, 32768, 65536 * 3]],
                        [[1, 1, -1, 5, 9, 2 ** 25, 2 ** 30, 7]]], dtype=torch.int32)
    out, l, flags = run(c, q, block_ids=ids, lists=1)
    assert flags == 0
    keep = torch.tensor([[[2, 0]], [[-1, -1]]], dtype=torch.int32)
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5, keep, 1))


@pytest.mark.parametrize("dtype", DTYPES)
def test_lists_of_every_block_are_the_whole_cache(dtype):
    lens = [drafts(L, 2) for L in (1, 500, 1025)]
    c = _attn.make(dtype, lens, 1, 61)
    q = draws(3, 2, 8, 11)
    ids = torch.arange(9, dtype=torch.int32).flip(0).expand(3, 4, 9).contiguous()
    ref = _attn.reference(c, q, 128 ** -0.5)
    out, l, _ = run(c, q, block_ids=ids, lists=2)
    _attn.check(out, l, ref)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_token_that_one_draft_row_sees_does_not_reach_the_others(dtype, bad):
    """The rows of a unit share one product with the values: 0 * NaN must not leak."""
    lens = [drafts(130, 4), drafts(64, 4)]
    c = _attn.make(dtype, lens, 1, 71)
    clean = _attn.reference(c, draws(2, 4, 4, 12), 128 ** -0.5)
    page = c.page_table[int(c.slot_ids[0])]
    row = int(page[129 // 64]) * 64 + 129 % 64        # the newest token: only the last row sees it
    if dtype == "bf16":
        c.v[0][row, 5] = bad
        c.k[0][row, 3] = bad
    else:
        c.v[1][row] = bad
        c.k[1][row] = bad
    q = draws(2, 4, 4, 12)
    out, l, flags = run(c, q)
    assert flags == 0
    out, l = out.cpu(), l.cpu()
    keep = torch.ones((2, 4, 4), dtype=torch.bool)
    keep[0, 3] = False
    d = (out.double() - clean[0]).abs()
    assert (d[keep] <= clean[2][keep]).all()
    assert ((l.double() - clean[1]).abs()[keep] <= clean[3][keep]).all()
    if bad != -float("inf"):
        # a NaN or +inf score makes the row that sees it not finite (-inf may be a weight of zero)
        assert not torch.isfinite(out[0, 3].float()).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_block_that_one_draft_row_lists_does_not_reach_the_others(dtype):
    lens = [[640, 640]]
    c = _attn.make(dtype, lens, 1, 73)
    ids = torch.tensor([[[0, 1, 2], [0, 3, 2]]], dtype=torch.int32)
    q = draws(1, 2, 4, 13)
    clean = _attn.reference(c, q, 128 ** -0.5, ids, 1)
    page = c.page_table[int(c.slot_ids[0])]
    row = int(page[3 * 128 // 64]) * 64 + 7            # in block 3
    if dtype == "bf16":
        c.v[0][row] = float("nan")
    else:
        c.v[0][row] = 0x7f
    out, l, _ = run(c, q, block_ids=ids, lists=1)
    d = (out.cpu().double() - clean[0]).abs()
    assert (d[0, 0] <= clean[2][0, 0]).all()
    assert torch.isnan(out[0, 1].float()).all()
    assert ((l.cpu().double() - clean[1]).abs() <= clean[3]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_far_apart_and_value_scales_far_apart(dtype):
    """A running maximum that grows late, weights that vanish, values over many powers of two."""
    lens = [drafts(900, 2)]
    c = _attn.make(dtype, lens, 1, 81, spread=True)
    q = draws(1, 2, 8, 14, scale=40.0)
    out, l, flags = run(c, q)
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


def test_zero_scales_and_zero_queries():
    lens = [[200]]
    c = _attn.make("fp8_e4m3", lens, 1, 83)
    c.v[1].zero_()
    q = draws(1, 1, 4, 15)
    q[:, :, 1] = 0
    out, l, _ = run(c, q)
    assert torch.equal(out, torch.zeros_like(out))
    ref = _attn.reference(c, q, 128 ** -0.5)
    assert ((l.cpu().double() - ref[1]).abs() <= ref[3]).all()


def test_no_lse_and_no_requests():
    c = _attn.make("bf16", [[100]], 1, 85)
    q = draws(1, 1, 4, 16)
    a, l, _ = run(c, q)
    b, none, _ = run(c, q, lse=False)
    assert none is None and torch.equal(a, b)
    d = _attn.to_device(c)
    ws = idx.alloc_attn_workspace(1, 4, 1)
    ws.fill_(0xff)
    idx.idx_attn_paged(q[:0].cuda(), d.k[0], None, d.v[0], None, "bf16", d.page_table,
                       d.slot_ids[:0], d.row_lens[:0], 1, 1.0, a[:0], None, ws)
    assert idx.idx_workspace_errors(ws) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("blocks", [False, True])
def test_bad_pages_are_left_out_and_flagged(dtype, blocks):
    lens = [[500], [300]]
    c = _attn.make(dtype, lens, 2, 87)
    s = int(c.slot_ids[0])
    c.page_table[s, 2] = c.num_pages           # past the pool
    c.page_table[s, 5] = -3
    q = draws(2, 1, 4, 17)
    ids = torch.arange(4, dtype=torch.int32).expand(2, 1, 4).contiguous() if blocks else None
    out, l, flags = run(c, q, block_ids=ids, lists=1 if blocks else 0)
    assert flags == idx._lib.DEVERR_BAD_PAGE
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5, ids, 1))


def test_lengths_past_the_table_are_clamped_and_flagged():
    c = _attn.make("bf16", [[200], [90]], 1, 89, max_pages=4)
    c.row_lens[0] = 100000
    c.page_table[int(c.slot_ids[0])] = torch.arange(4, dtype=torch.int32)
    c.k[0].nan_to_num_(0.5)
    c.v[0].nan_to_num_(0.5)
    q = draws(2, 1, 4, 18)
    out, l, flags = run(c, q)
    assert flags == idx._lib.DEVERR_LEN_CLAMPED
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


def test_negative_lengths_are_empty_rows():
    c = _attn.make("bf16", [[200, 100]], 1, 91)
    c.row_lens[0, 1] = -5
    q = draws(1, 2, 4, 19)
    out, l, _ = run(c, q)
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


def test_planes_past_32_bit_offsets():
    """Pages near the end of 5 GB planes."""
    pages, H = 300_000, 1
    kp = torch.empty((pages * H * 64, 128), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    use = [pages - 1, pages - 7, 3, pages - 2]
    c = _attn.make("bf16", [[250]], H, 93, garbage=False)
    src = c.page_table[int(c.slot_ids[0])].tolist()
    for i, p in enumerate(use):
        kp[p * 64:(p + 1) * 64] = c.k[0][src[i] * 64:(src[i] + 1) * 64].cuda()
        vp[p * 64:(p + 1) * 64] = c.v[0][src[i] * 64:(src[i] + 1) * 64].cuda()
    q = draws(1, 1, 16, 20)
    out = torch.empty((1, 1, 16, 128), dtype=torch.bfloat16, device="cuda")
    l = torch.empty((1, 1, 16), device="cuda")
    ws = idx.alloc_attn_workspace(1, 16, 1)
    idx.idx_attn_paged(q.cuda(), kp, None, vp, None, "bf16",
                       torch.tensor([use], dtype=torch.int32, device="cuda"),
                       torch.zeros(1, dtype=torch.int32, device="cuda"),
                       torch.tensor([[250]], dtype=torch.int32, device="cuda"), H, 128 ** -0.5, out, l, ws)
    assert idx.idx_workspace_errors(ws) == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


def test_graph_replay_and_another_stream():
    lens = [drafts(L, 2) for L in (900, 64)]
    c = _attn.make("bf16", lens, 1, 95)
    q = draws(2, 2, 8, 21)
    want, wl, _ = run(c, q)
    d = _attn.to_device(c)
    qd = q.cuda()
    out, l = torch.zeros_like(want), torch.zeros_like(wl)
    ws = idx.alloc_attn_workspace(2, 8, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    idx.idx_attn_paged(qd, *d.args(), 1, 128 ** -0.5, out, l, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(l, wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx.idx_attn_paged(qd, *d.args(), 1, 128 ** -0.5, out, l, ws)
    d.row_lens[0] = torch.tensor([310, 311], dtype=torch.int32)
    graph.replay()
    torch.cuda.synchronize()
    c.row_lens[0] = torch.tensor([310, 311], dtype=torch.int32)
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P,Hq", [(1, 8), (4, 16)])
def test_a_wait_that_runs_out_is_flagged(dtype, P, Hq):
    c = _attn.make(dtype, [drafts(3000, P)], 1, 97)
    q = draws(1, P, Hq, 22)
    idx.idx_set_wait_limit_ns(20_000_000)
    idx.idx_set_stall_test(True)
    try:
        _, _, flags = run(c, q)
    finally:
        idx.idx_set_stall_test(False)
        idx.idx_set_wait_limit_ns(0)
    assert flags & idx._lib.DEVERR_TIMEOUT
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


def test_shards_join_by_lse():
    """Two halves of a context, joined by their lse, are the whole."""
    c = _attn.make("bf16", [[1024]], 1, 99, garbage=False)
    q = draws(1, 1, 8, 23)
    whole, wl, _ = run(c, q)
    parts = []
    table = c.page_table[int(c.slot_ids[0])].clone()
    for half in range(2):
        c.page_table[int(c.slot_ids[0]), :8] = table[8 * half:8 * half + 8]
        c.row_lens[0, 0] = 512
        parts.append(run(c, q)[:2])
    l = torch.stack([p[1] for p in parts])
    z = torch.logsumexp(l, 0)
    out = sum(p[0].float() * torch.exp(p[1] - z)[..., None] for p in parts)
    assert (z - wl).abs().max() <= 2e-5
    # each side: a bf16 rounding of the weights and of the result
    assert (out - whole.float()).abs().max() <= 2 * 2.0 ** -8 * whole.float().abs().max() + 2.0 ** -8


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P,Hq", [(1, 16), (4, 16), (4, 32)])
def test_one_long_request_over_many_parts(dtype, P, Hq):
    """One unit over every CTA: the join of a hundred parts a row."""
    c = _attn.make(dtype, [drafts(20011, P)], 1, 101)
    q = draws(1, P, Hq, 24)
    out, l, flags = run(c, q)
    again, l2, _ = run(c, q)
    assert flags == 0 and torch.equal(out, again) and torch.equal(l, l2)
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P,Hq,Hkv", [(1, 4, 2), (6, 4, 1)])
def test_many_short_requests(dtype, P, Hq, Hkv):
    """More requests than the threads that read them, several units a CTA."""
    g = torch.Generator().manual_seed(3)
    lens = [drafts(int(L), P) for L in torch.randint(0, 90, (700,), generator=g)]
    c = _attn.make(dtype, lens, Hkv, 103, pads=(0, 255, 256, 699))
    q = draws(700, P, Hq, 25)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


@pytest.mark.parametrize("blocks", [False, True])
def test_page_tables_so_wide_that_pieces_are_counted_in_lots(blocks):
    """The line of positions is kept short by counting pieces two at a time."""
    R, P = (64, 1) if not blocks else (150, 16)
    lens = [drafts(L, P) for L in ([900, 65, 0, 31] * 64)[:R]]
    c = _attn.make("bf16", lens, 2, 105, max_pages=65536 if not blocks else 20000)
    q = draws(R, P, 4, 26)
    ids = lists_for(lens, 2, 256, 27, P) if blocks else None
    out, l, flags = run(c, q, block_ids=ids, lists=2 if blocks else 0)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ctas", [3, 0])
def test_blocks_of_wide_units(dtype, ctas):
    """Block lists with more than 16 rows a unit, several units a CTA."""
    P = 4
    lens = [drafts(L, P) for L in (3000, 0, 129, 4096, 64, 2049)]
    c = _attn.make(dtype, lens, 2, 107, pads=(4,))
    q = draws(len(lens), P, 16, 28)
    ids = lists_for(lens, 2, 7, 29, P)
    idx.idx_set_grid_limit(ctas)
    try:
        out, l, flags = run(c, q, block_ids=ids, lists=2)
    finally:
        idx.idx_set_grid_limit(0)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5, ids, 2))


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_far_apart_with_many_rows(dtype):
    """The wide kernel's late raises of the running maximum, and values over many scales."""
    c = _attn.make(dtype, [drafts(1500, 4)], 1, 109, spread=True)
    q = draws(1, 4, 16, 30, scale=40.0)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_one_draft_rows_token_among_many_rows(dtype, bad):
    """As the narrow test: the newest token is not finite, only the last draft row sees it."""
    lens = [drafts(200, 4), drafts(65, 4)]
    c = _attn.make(dtype, lens, 1, 111)
    q = draws(2, 4, 16, 31)
    clean = _attn.reference(c, q, 128 ** -0.5)
    page = c.page_table[int(c.slot_ids[0])]
    row = int(page[199 // 64]) * 64 + 199 % 64
    for p in (c.k, c.v):
        if dtype == "bf16":
            p[0][row] = bad
        else:
            p[1][row] = bad
    out, l, flags = run(c, q)
    assert flags == 0
    keep = torch.ones((2, 4, 16), dtype=torch.bool)
    keep[0, 3] = False
    d = (out.cpu().double() - clean[0]).abs()
    assert (d[keep] <= clean[2][keep]).all()
    assert ((l.cpu().double() - clean[1]).abs()[keep] <= clean[3][keep]).all()
    assert not torch.isfinite(out[0, 3].float()).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_native_call_and_the_python_one_agree(dtype):
    from sparse_attention_indexer_packed_gb300 import _lib
    assert idx.idx_attn_paged is not _lib.idx_attn_paged, "the CPython module has not been built"
    lens = [drafts(L, 2) for L in (300, 77)]
    c = _attn.to_device(_attn.make(dtype, lens, 1, 113))
    q = draws(2, 2, 4, 32).cuda()
    ids = torch.tensor([[[0, 2], [1, 2]] * 2] * 2, dtype=torch.int32, device="cuda")
    ws = idx.alloc_attn_workspace(2, 4, 1, 2)
    scale = 128 ** -0.5
    got = []
    for paged, blocks in ((idx.idx_attn_paged, idx.idx_attn_blocks), (_lib.idx_attn_paged, _lib.idx_attn_blocks)):
        out, l = torch.empty_like(q), torch.empty((2, 2, 4), device="cuda")
        paged(q, *c.args(), 1, scale, out, l, ws)
        got.append((out.clone(), l.clone()))
        paged(q, *c.args(), kv_heads=1, sm_scale=scale, out=out, out_lse=None, workspace=ws)
        assert torch.equal(out, got[-1][0])
        blocks(q, *c.args(), ids, 2, 1, scale, out, l, ws)
        got.append((out.clone(), l.clone()))
        good = (q, *c.args(), 1, scale, out, l, ws)
        for at, bad in ((0, q.float()), (0, q[..., :64]), (0, q.transpose(1, 2)), (1, c.k[0][:65]),
                        (6, c.page_table.long()), (7, c.slot_ids[:1]), (8, c.row_lens.t()), (9, 3),
                        (10, -1.0), (11, out[:1]), (12, l.double()), (13, ws[:1024]), (13, ws.cpu()),
                        (5, "int8")):
            with pytest.raises(idx.IdxError):
                paged(*good[:at], bad, *good[at + 1:])
        good = (q, *c.args(), ids, 2, 1, scale, out, l, ws)
        for at, bad in ((9, ids[:, :3]), (9, ids.long()), (9, None), (10, 3), (10, 0)):
            with pytest.raises(idx.IdxError):
                blocks(*good[:at], bad, *good[at + 1:])
    for a, b in ((0, 2), (1, 3)):
        assert torch.equal(got[a][0], got[b][0]) and torch.equal(got[a][1], got[b][1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq", [4, 16])
def test_rows_that_see_nothing_but_nan_are_nan(dtype, Hq):
    """Not mistaken for rows that see nothing: a request of one token, one of 200, all NaN."""
    lens = [drafts(1, 4), drafts(200, 4), drafts(90, 4)]
    c = _attn.make(dtype, lens, 1, 115)
    q = draws(3, 4, Hq, 33)
    clean = _attn.reference(c, q, 128 ** -0.5)
    for r, n in ((0, 1), (1, 200)):
        rows = _attn.token_rows(c.page_table[int(c.slot_ids[r])].tolist(), n, 0, 1)
        (c.k[0] if dtype == "bf16" else c.k[1])[rows] = float("nan")
    out, l, flags = run(c, q)
    assert flags == 0
    out, l = out.cpu().float(), l.cpu()
    for r in range(2):
        for p in range(4):
            if lens[r][p] > 0:
                assert torch.isnan(out[r, p]).all() and torch.isnan(l[r, p]).all()
            else:
                assert (out[r, p] == 0).all() and torch.isinf(l[r, p]).all()
    assert ((out[2].double() - clean[0][2]).abs() <= clean[2][2]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("blocks,Hq,more", [(False, 4, 0), (True, 4, 0), (True, 2, 0), (False, 1, 40)])
def test_many_draft_rows(dtype, blocks, Hq, more):
    """A chunk of 70 tokens a request, each with its own length; few requests, and many."""
    P = 70
    lens = [drafts(L, P) for L in [300, 40, 0, 129] + list(range(more))]
    c = _attn.make(dtype, lens, 1, 117)
    q = draws(len(lens), P, Hq, 34)
    ids = lists_for(lens, 2, 3, 35, P) if blocks else None
    out, l, flags = run(c, q, block_ids=ids, lists=2 if blocks else 0)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5, ids, 2))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,Hkv", [(2, 1), (5, 1), (3, 4), (23, 1), (10, 4), (67, 2)])
def test_many_short_requests_on_few_ctas(dtype, R, Hkv):
    """Units that warps, pairs, fours and whole CTAs take, in one turn and in several; the last
    row of request 1 sees a NaN that its other rows do not."""
    lens = [drafts(L % 190, 3) for L in range(1, 37 * R, 37)]
    lens[1] = drafts(40, 3)
    c = _attn.make(dtype, lens, Hkv, 121, pads=(4,) if R > 4 else ())
    q = draws(R, 3, 2 * Hkv, 36)
    ref = _attn.reference(c, q, 128 ** -0.5)
    rows = _attn.token_rows(c.page_table[int(c.slot_ids[1])].tolist(), 40, 0, Hkv)
    (c.v[0] if dtype == "bf16" else c.v[1])[rows[-1]] = float("nan")
    idx.idx_set_grid_limit(4)
    try:
        out, l, flags = run(c, q)
        again, l2, _ = run(c, q)
    finally:
        idx.idx_set_grid_limit(0)
    assert flags == 0
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(l, l2)
    assert torch.isnan(out[1, 2, :2].float()).all()
    out[1, 2, :2] = ref[0][1, 2, :2].to(out)
    _attn.check(out, l, ref)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,lists,topk", [(5, 1, 3), (3, 2, 9), (7, 2, 5), (20, 2, 4), (9, 1, 256)])
def test_many_short_lists_on_few_ctas(dtype, R, lists, topk):
    """The same with block lists, each team joining its own."""
    lens = [drafts(97 * k % 2900, 4) for k in range(R)]
    c = _attn.make(dtype, lens, 1, 123, pads=(1,))
    q = draws(R, 4, 2 * lists, 37)
    ids = lists_for(lens, lists, topk, 38, 4)
    idx.idx_set_grid_limit(4)
    try:
        out, l, flags = run(c, q, block_ids=ids, lists=lists)
        again, l2, _ = run(c, q, block_ids=ids, lists=lists)
    finally:
        idx.idx_set_grid_limit(0)
    assert flags == 0
    assert torch.equal(out, again) and torch.equal(l, l2)
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5, ids, lists))


@pytest.mark.parametrize("Hq", [1, 4, 12])
@pytest.mark.parametrize("blocks", [False, True])
def test_value_scales_of_tokens_a_row_does_not_see(Hq, blocks):
    """A row's precision does not depend on the tokens of the other rows: the last token, or
    the other list's blocks, have values 2^24 times larger."""
    P = 3
    lens = [drafts(L, P) for L in (4, 40, 300, 257)]
    c = _attn.make("fp8_e4m3", lens, 1, 125)
    for r, row in enumerate(lens):
        rows = _attn.token_rows(c.page_table[int(c.slot_ids[r])].tolist(), max(row), 0, 1)
        c.v[1][rows[-1]] *= 2.0 ** 24
        if blocks and max(row) > 128:
            c.v[1][rows[:128]] *= 2.0 ** 24
    q = draws(4, P, Hq, 39)
    ids = None
    if blocks:
        ids = torch.full((4, P, 2), -1, dtype=torch.int32)
        for r, row in enumerate(lens):
            last = (max(row) - 1) // 128
            ids[r, 0, 0] = ids[r, 1, 1] = 0 if last == 0 else 1     # not block 0, where there is another
            ids[r, 2, 0] = last
            ids[r, 2, 1] = 0
    out, l, flags = run(c, q, block_ids=ids, lists=1 if blocks else 0)
    assert flags == 0
    _attn.check(out, l, _attn.reference(c, q, 128 ** -0.5, ids, 1))
