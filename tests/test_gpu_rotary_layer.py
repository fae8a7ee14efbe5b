"""The example layer with normed and turned queries and keys (needs a GPU): the pass that norms,
turns and stores, the index step over what it left, block and whole-cache attention, over every
type of cache; eager and captured."""
import pytest
import torch

import _attn
import _nvfp4
from test_gpu_example import example

pytestmark = pytest.mark.gpu
HIDDEN, HQ, G, TOPK = 256, 8, 4, 6


def setup(kv_dtype, drafts, kv_heads, axes):
    """A layer whose caches hold requests of several lengths, and a step's arguments."""
    R, L = 3, 1900
    layer = example().SparseDecodeLayer(hidden=HIDDEN, q_heads=HQ, kv_heads=kv_heads, index_heads=G, topk=TOPK,
                                        max_requests=R, max_tokens=L + 64, drafts=drafts, kv_dtype=kv_dtype,
                                        rotary=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda n: torch.randn((n, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    lens = torch.tensor([L, 130, drafts], dtype=torch.int32, device="cuda")
    for r, n in enumerate((lens - drafts).tolist()):
        pos = torch.arange(n, device="cuda")
        layer.write(rand(n), rand(n), layer.slots(torch.full_like(pos, r), pos), axes_of(pos, axes))
    request = torch.arange(R, dtype=torch.int32, device="cuda")
    at = (lens[:, None] - drafts + torch.arange(drafts, dtype=torch.int32, device="cuda")).reshape(-1)
    return layer, request, lens, at, rand


def axes_of(pos, axes):
    """Positions of tokens in a picture 40 wide of 12 rows a frame, or along the text."""
    if axes == 1:
        return pos.int()
    return torch.stack([pos // 480, pos // 40 % 12, pos % 40]).int()


def cache(layer, request, lens, drafts):
    cpu = lambda p: tuple(None if t is None else t.cpu() for t in p)  # noqa: E731
    rows = lens.cpu()[:, None] - drafts + 1 + torch.arange(drafts)
    return _attn.Cache(layer.kv_dtype, layer.kv_heads, layer.page_table.numel(), cpu(layer.k), cpu(layer.v),
                       layer.page_table.cpu(), request.cpu(), rows.to(torch.int32))


def reference(c, q, ids=None):
    make = _nvfp4.reference if c.dtype == "nvfp4" else _attn.reference
    return make(c, q, 128 ** -0.5, ids, G if ids is not None else 0)


def turned64(layer, x, weight, pos):
    x = x.double()
    x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double().cpu()
    i = torch.arange(64)
    p = pos.cpu().long()
    p = p[:, None].expand(-1, 64) if p.dim() == 1 else p[torch.tensor(list(layer.pair_axis))].T
    t = layer.table.cpu().double()
    c, s = t[p, i][:, None], t[p, 64 + i][:, None]
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("kv_dtype,drafts,kv_heads,axes", [
    ("nvfp4", 1, 2, 1), ("nvfp4", 4, 1, 1), ("nvfp4", 8, 1, 3), ("bf16", 1, 2, 3), ("fp8_e4m3", 4, 1, 1)])
def test_step(kv_dtype, drafts, kv_heads, axes):
    layer, request, lens, at, rand = setup(kv_dtype, drafts, kv_heads, axes)
    R = len(lens)
    x, res, pos = rand(R * drafts), rand(R * drafts), axes_of(at, axes)
    out, lse, _, ids = layer.step(x, res, request, lens, positions=pos)
    c = cache(layer, request, lens, drafts)
    parts, _ = layer.write(x, res, layer.slots(request.long().repeat_interleave(drafts), at.long()), pos)
    # (bytes: rows that nothing was written to hold anything)
    assert all(torch.equal(a.view(torch.uint8), b.cpu().view(torch.uint8)) for a, b in zip(c.k, layer.k)
               if a is not None)
    q = parts[0].reshape(R, drafts, HQ, 128).cpu()
    _attn.check(out, lse, reference(c, q, ids.cpu()))
    full, full_lse, _, _ = layer.step(x, res, request, lens, sparse=False, positions=pos)
    _attn.check(full, full_lse, reference(c, q))
    # requests that fit their lists attend to everything they have
    assert torch.allclose(lse[1:].cpu(), full_lse[1:].cpu(), atol=1e-4)
    # the blocks of the longest request: the index queries and keys as the formulas have them.
    # The keys are read as stored, a query's code is off by 2^-4 of its element, or by 2^-19 of the
    # row's largest: a score by less than 2^-3 of |q| |k|.  A block that is listed scores no lower,
    # by that, than one that is not
    raw, _ = raw_parts(layer, x, res)
    iq = turned64(layer, raw[3].cpu(), layer.index_norm, pos).reshape(R, drafts * G, 128)
    t = torch.arange(int(lens[0]))
    rows = (layer.page_table[0].cpu().long()[t // 64] * 64 + t % 64)
    codes, scale = (p.cpu()[rows] for p in layer.index_keys)
    ik = codes.view(torch.float8_e4m3fn).double() * scale.double()
    for m in range(drafts * G):
        n = int(lens[0]) - drafts + 1 + m // G
        s, e = ik[:n] @ iq[0, m], (ik[:n].abs() @ iq[0, m].abs()) * 2.0 ** -3
        block = t[:n] // 128
        blocks = int(block[-1]) + 1
        low, high = (torch.stack([v[block == b].max() for b in range(blocks)]) for v in (s - e, s + e))
        free = torch.ones(blocks, dtype=torch.bool)
        free[:layer.init_blocks] = free[-layer.local_blocks:] = False
        listed = torch.zeros(blocks, dtype=torch.bool)
        listed[ids[0, m][ids[0, m] >= 0].cpu().long()] = True
        assert listed[~free].all() and int(listed.sum()) == TOPK
        assert high[free & listed].min() >= low[free & ~listed].max()


def raw_parts(layer, x, res):
    """The projection before norm and rotation."""
    table, layer.table = layer.table, None
    keep = layer.k, layer.v, layer.index_keys
    layer.k, layer.v, layer.index_keys = (tuple(None if t is None else t.clone() for t in p) for p in keep)
    try:
        return layer.write(x, res, torch.full((len(x),), -1, device="cuda"))
    finally:
        layer.table, (layer.k, layer.v, layer.index_keys) = table, keep


@pytest.mark.parametrize("sparse", [True, False])
def test_captured_step(sparse):
    """A step's calls in one graph, replayed with other tokens and lengths: the eager step's bytes."""
    drafts = 2
    layer, request, lens, at, rand = setup("nvfp4", drafts, 1, 1)
    R = len(lens)
    x, res, n = rand(R * drafts), rand(R * drafts), lens.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step(x, res, request, n, sparse)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(x, res, request, n, sparse)
    for k in range(3):
        x.copy_(rand(R * drafts))
        res.copy_(rand(R * drafts))
        n.copy_(lens + k)
        graph.replay()
        out, lse = got[0].clone(), got[1].clone()
        want = layer.step(x, res, request, n, sparse)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        c = cache(layer, request, n, drafts)
        rows = n[:, None] - drafts + torch.arange(drafts, dtype=torch.int32, device="cuda")
        parts, _ = layer.write(x, res, layer.slots(request[:, None].long(), rows.long()).reshape(-1), rows.reshape(-1))
        _attn.check(out, lse, reference(c, parts[0].reshape(R, drafts, HQ, 128).cpu(),
                                        want[3].cpu() if sparse else None))


def test_main_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["x", "--requests", "2", "--context", "900", "--steps", "1", "--kv-dtype",
                                     "nvfp4", "--rotary"])
    example().main()
    assert "of the attention weight" in capsys.readouterr().out
