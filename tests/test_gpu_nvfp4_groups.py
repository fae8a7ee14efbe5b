"""Attention over an NVFP4 cache (needs a GPU): more draft rows than one group of rows holds, calls
without a log-sum, and a captured call over block lists."""
import pytest
import torch

import _attn
import _nvfp4
import sparse_attention_indexer_packed_gb300 as idx
from test_gpu_attn import drafts, draws, lists_for
from test_gpu_nvfp4 import SCALE, TABLES, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_pages", TABLES)      # (groups of 16 rows, of 128)
@pytest.mark.parametrize("P,Hq,Hkv", [(20, 16, 1), (130, 2, 1), (9, 30, 2), (1, 300, 1)])
def test_several_groups(P, Hq, Hkv, max_pages):
    lens = [drafts(L, P) for L in (700, 0, 64, 129, 5, 1030)]
    lens[3][P // 2] = 0
    c = _nvfp4.make(lens, Hkv, 301 + P, pads=(4,), max_pages=max_pages)
    q = draws(len(lens), P, Hq, 71)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE))


@pytest.mark.parametrize("more", [0, 200])
@pytest.mark.parametrize("P,Hq,Hkv,lists", [(40, 4, 1, 1), (35, 6, 2, 2), (3, 400, 1, 2), (33, 16, 1, 16)])
def test_several_groups_of_block_lists(P, Hq, Hkv, lists, more):
    lens = [drafts(L, P) for L in (700, 0, 64, 1300, 130)]
    c = _nvfp4.make(lens, Hkv, 311 + P, pads=(2,), max_pages=4000 if more else None)
    q = draws(len(lens), P, Hq, 72)
    ids = lists_for(lens, lists, 6, 73, P)
    ids[3, P * lists // 2] = -1
    ids = torch.cat([ids, torch.full((*ids.shape[:2], more), -1, dtype=torch.int32)], 2)
    out, l, flags = run(c, q, block_ids=ids, lists=lists)
    assert flags == 0
    _attn.check(out, l, _nvfp4.reference(c, q, SCALE, ids, lists))


@pytest.mark.parametrize("max_pages", TABLES)
@pytest.mark.parametrize("P,Hq,lists", [(1, 8, 0), (4, 16, 0), (2, 8, 2), (4, 32, 1)])
def test_without_a_log_sum(P, Hq, lists, max_pages):
    lens = [drafts(L, P) for L in (900, 70, 0)]
    c = _nvfp4.make(lens, 1, 321, max_pages=max_pages)
    q = draws(3, P, Hq, 74)
    ids = lists_for(lens, lists, 5, 75, P) if lists else None
    out, _, _ = run(c, q, block_ids=ids, lists=lists)
    alone, l, flags = run(c, q, block_ids=ids, lists=lists, lse=False)
    assert flags == 0 and l is None and torch.equal(out, alone)


@pytest.mark.parametrize("P,Hq", [(2, 8), (4, 16)])
def test_two_graphs_that_share_a_workspace(P, Hq):
    """Captured on one stream, replayed in either order with new queries and lists."""
    lens = [drafts(L, P) for L in (1500, 90)]
    c = _nvfp4.make(lens, 1, 331)
    d = _attn.to_device(c)
    q = draws(2, P, Hq, 76).cuda()
    ids = lists_for(lens, 2, 6, 77, P).cuda()
    out = [torch.empty_like(q) for _ in range(2)]
    l = [torch.empty((2, P, Hq), device="cuda") for _ in range(2)]
    ws = idx.alloc_attn_workspace(P, Hq, 1, 2)
    head = (q, *d.k, *d.v, d.page_table, d.slot_ids, d.row_lens)
    calls = (lambda: idx.idx_attn_paged_nvfp4(*head, 1, SCALE, out[0], l[0], ws),
             lambda: idx.idx_attn_blocks_nvfp4(*head, ids, 2, 1, SCALE, out[1], l[1], ws))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for f in calls:
            f()
    s.synchronize()
    graphs = []
    for f in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for order, seed in (((0, 1), 78), ((1, 0), 79)):
        new, lists = draws(2, P, Hq, seed), lists_for(lens, 2, 6, seed, P)
        q.copy_(new)
        ids.copy_(lists)
        for i in order:
            graphs[i].replay()
        assert idx.idx_workspace_errors(ws) == 0
        _attn.check(out[0], l[0], _nvfp4.reference(c, new, SCALE))
        _attn.check(out[1], l[1], _nvfp4.reference(c, new, SCALE, lists, 2))
