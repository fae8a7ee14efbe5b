"""Attention over an NVFP4 cache (needs a GPU) where the split of the work takes its rarer ways:
block lists dealt whole to teams of a CTA's warps, pieces counted in lots, more row groups than
one kernel takes, and a NaN that one draft row of a unit lists."""
import dataclasses

import pytest
import torch

import _attn
import _nvfp4
import sparse_attention_indexer_packed_gb300 as idx
from test_gpu_attn import drafts, draws, lists_for
from test_gpu_nvfp4 import SCALE, run

pytestmark = pytest.mark.gpu


def ragged(R, P, longest, seed):
    g = torch.Generator().manual_seed(seed)
    return [drafts(int(n), P) for n in torch.randint(0, longest + 1, (R,), generator=g)]


# On 152 SMs a unit goes to 12 warps up to 152 units, to 6 up to 304, else to 3; with a limit on
# the CTAs a team takes several units in turn.  min(P, 16) * topk is 1024 and 2048 in the last
# three: all that the joined list of 3 or of 6 warps holds.
@pytest.mark.parametrize("R,P,Hq,Hkv,lists,topk,ctas", [
    (70, 1, 16, 1, 4, 8, 0), (64, 4, 8, 1, 4, 5, 0), (100, 1, 8, 2, 2, 16, 0), (45, 2, 8, 1, 4, 3, 7),
    (110, 1, 16, 1, 4, 16, 0), (130, 2, 8, 2, 4, 3, 0), (300, 1, 4, 1, 2, 6, 0), (24, 4, 8, 1, 4, 6, 2),
    (20, 4, 8, 1, 4, 5, 1), (64, 4, 8, 2, 2, 256, 7), (20, 4, 8, 2, 2, 256, 7), (20, 8, 8, 2, 2, 256, 7)])
def test_block_lists_dealt_whole_to_teams(R, P, Hq, Hkv, lists, topk, ctas):
    lens = ragged(R, P, 900 if topk < 256 else 2000, R + topk)
    pads = (0, R // 2, R - 1)
    c = _nvfp4.make(lens, Hkv, 201 + R, pads=pads)
    q = draws(R, P, Hq, 61)
    ids = lists_for(lens, lists, topk, 62, P)
    ids[1, 0, 0] = ids[1, 0, topk // 2]      # a block twice, none, and one past the row's own
    ids[2, 0, -1] = -3
    ids[3, P * lists - 1, topk // 2] = 40
    idx.idx_set_grid_limit(ctas)
    try:
        out, l, flags = run(c, q, block_ids=ids, lists=lists)
        again, l2, _ = run(c, q, block_ids=ids, lists=lists)
    finally:
        idx.idx_set_grid_limit(0)
    assert flags == 0
    assert torch.equal(out, again) and torch.equal(l, l2)
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE, ids, lists))


@pytest.mark.parametrize("P,Hq", [(1, 4), (20, 4)])
def test_pieces_counted_in_lots(P, Hq):
    """64 requests x 2 key heads x 65536 pages: more half-page pieces than the line has positions."""
    lens = [drafts(L, P) for L in [900, 65, 0, 31, 2100, 130, 64, 1] * 8]
    c = _nvfp4.make(lens, 2, 211, pads=(5,), max_pages=65536)
    q = draws(len(lens), P, Hq, 63)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


@pytest.mark.parametrize("Hq", [8, 24])
def test_listed_pieces_counted_in_lots(Hq):
    """100 requests x 8 lists x 16 draft rows of 256 blocks, up to 16 and up to 48 rows a unit."""
    R, P, lists = 100, 16, 8
    lens = [drafts(L, P) for L in ([1700, 0, 65, 0, 31, 0, 300, 0, 0, 0] * R)[:R]]
    c = _nvfp4.make(lens, 2, 213, max_pages=20000)
    q = draws(R, P, Hq, 64)
    ids = lists_for(lens, lists, 256, 65, P)
    ids[..., 6:] = -1
    out, l, flags = run(c, q, block_ids=ids, lists=lists)
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE, ids, lists))


def many(c, R):
    """The batch repeated up to R requests, and a copy with some of them for the reference."""
    n = len(c.slot_ids)
    at = torch.arange(R) % n
    big = dataclasses.replace(c, slot_ids=c.slot_ids[at], row_lens=c.row_lens[at])
    pick = torch.tensor([0, 1, 2, R // 2, R - 2, R - 1])
    return big, dataclasses.replace(c, slot_ids=big.slot_ids[pick], row_lens=big.row_lens[pick]), pick


def test_more_row_groups_than_the_kernel_of_16_rows_takes():
    """17 rows a unit and 2048 x 65 units: two groups of 16 rows each would be past 2^18."""
    R, P, H = 2048, 17, 65
    c = _nvfp4.make([drafts(L, P) for L in (130, 64, 0, 17, 200, 3, 65, 128)], H, 215, pads=(3,))
    big, some, pick = many(c, R)
    d = _attn.to_device(big)
    g = torch.Generator(device="cuda").manual_seed(66)
    q = torch.randn((R, P, H, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    out, l = torch.full_like(q, 7.0), torch.full((R, P, H), 7.0, device="cuda")
    ws = idx.alloc_attn_workspace(P, H, H)
    idx.idx_attn_paged_nvfp4(q, *d.k, *d.v, d.page_table, d.slot_ids, d.row_lens, H, SCALE, out, l, ws)
    assert idx.idx_workspace_errors(ws) == 0
    pick = pick.cuda()
    _attn.check(out[pick], l[pick], _nvfp4.reference(some, q[pick].cpu(), SCALE))


def test_units_so_many_that_their_ends_count_less_on_the_line():
    """2048 x 44 lists of four draft rows: a unit's end cannot take four times its positions."""
    R, P, lists, topk = 2048, 4, 44, 2
    lens = [drafts(L, P) for L in (130, 64, 0, 300, 200, 3, 65, 128)]
    c = _nvfp4.make(lens, 1, 217, pads=(3,))
    big, some, pick = many(c, R)
    d = _attn.to_device(big)
    g = torch.Generator(device="cuda").manual_seed(67)
    q = torch.randn((R, P, lists, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = lists_for(lens, lists, topk, 68, P)
    ids = ids[torch.arange(R) % len(lens)]
    out, l = torch.full_like(q, 7.0), torch.full((R, P, lists), 7.0, device="cuda")
    ws = idx.alloc_attn_workspace(P, lists, 1, lists)
    idx.idx_attn_blocks_nvfp4(q, *d.k, *d.v, d.page_table, d.slot_ids, d.row_lens, ids.cuda(), lists, 1, SCALE,
                              out, l, ws)
    assert idx.idx_workspace_errors(ws) == 0
    _attn.check(out[pick.cuda()], l[pick.cuda()],
                _nvfp4.reference(some, q[pick.cuda()].cpu(), SCALE, ids[pick], lists))


@pytest.mark.parametrize("R,Hq,topk", [(1, 4, 3), (1, 16, 3), (8, 32, 256)])   # (the last: above 16 rows a group)
def test_a_block_that_one_draft_row_lists_does_not_reach_the_others(R, Hq, topk):
    lens = [[640, 640]] * R
    ids = torch.full((R, 2, topk), -1, dtype=torch.int32)
    ids[:, 0, :3], ids[:, 1, :3] = torch.tensor([0, 1, 2]), torch.tensor([0, 3, 2])
    q = draws(R, 2, Hq, 69)
    for plane in ("k", "v"):
        c = _nvfp4.make(lens, 1, 219, max_pages=4000)
        clean = _nvfp4.reference(c, q, SCALE, ids, 1)
        row = int(c.page_table[int(c.slot_ids[0]), 3 * 128 // 64]) * 64 + 7       # in block 3
        getattr(c, plane)[1][row, 2] = 0x7f
        out, l, flags = run(c, q, block_ids=ids, lists=1)
        assert flags == 0
        seen = torch.isnan(out[0, 1].float()).cpu()
        assert seen.all() if plane == "k" else (seen[:, 32:48].all() and not seen[:, :32].any() and not seen[:, 48:].any())
        out[0, 1], l[0, 1] = clean[0][0, 1].to(out), clean[1][0, 1].to(l)
        _attn.check(out, l, clean)
