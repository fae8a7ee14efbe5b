"""The example layer's step (needs a GPU): norm, store, index step and block attention together,
each checked against plain arithmetic on what the step before it left."""
import importlib.util
import os

import pytest
import torch

import _attn

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("sparse_decode_layer",
                                                  os.path.join(ROOT, "examples", "sparse_decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kv_dtype,drafts,kv_heads", [("bf16", 1, 2), ("fp8_e4m3", 4, 1)])
def test_step(kv_dtype, drafts, kv_heads):
    ex = example()
    R, L = 3, 2100
    layer = ex.SparseDecodeLayer(hidden=512, q_heads=8, kv_heads=kv_heads, index_heads=4, topk=6,
                                 max_requests=R, max_tokens=L + 64, drafts=drafts, kv_dtype=kv_dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda n: torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    lens = torch.tensor([L, 130, 7], dtype=torch.int32, device="cuda")
    for r, n in enumerate((lens - drafts).tolist()):
        pos = torch.arange(n, device="cuda")
        layer.write(rand(n), rand(n), layer.slots(torch.full_like(pos, r), pos))
    request = torch.arange(R, dtype=torch.int32, device="cuda")
    x, res = rand(R * drafts), rand(R * drafts)
    out, lse, new, ids = layer.step(x, res, request, lens)
    assert torch.equal(new, (x.float() + res.float()).to(torch.bfloat16))
    # the attention over the ids that came out, from the cache as it lies now
    cpu = lambda p: tuple(None if t is None else t.cpu() for t in p)  # noqa: E731
    rows = lens.cpu()[:, None] - drafts + 1 + torch.arange(drafts)
    c = _attn.Cache(kv_dtype, kv_heads, layer.page_table.numel(), cpu(layer.k), cpu(layer.v),
                    layer.page_table.cpu(), request.cpu(), rows.to(torch.int32))
    parts, _ = layer.write(x, res, layer.slots(request[:, None].long(), (rows - 1).cuda()).reshape(-1))
    q = parts[0].reshape(R, drafts, 8, 128).cpu()
    _attn.check(out, lse, _attn.reference(c, q, 128 ** -0.5, ids.cpu(), 4))
    full, full_lse, _, none = layer.step(x, res, request, lens, sparse=False)
    assert none is None
    _attn.check(full, full_lse, _attn.reference(c, q, 128 ** -0.5))
    # a request that fits its list attends to everything it has
    assert torch.allclose(lse[1:].cpu(), full_lse[1:].cpu(), atol=1e-4)


def test_main_runs(capsys, monkeypatch):
    ex = example()
    monkeypatch.setattr("sys.argv", ["x", "--requests", "2", "--context", "900", "--steps", "1"])
    ex.main()
    assert "of the attention weight" in capsys.readouterr().out
