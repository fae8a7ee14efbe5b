"""Host-side checks of the key-value store, the attention and the norm (no compute call runs)."""
import ctypes

import pytest
import torch

import sparse_attention_indexer_packed_gb300 as idx
from sparse_attention_indexer_packed_gb300 import _lib

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return idx.lib()


def attn(L, blocks=False, **over):
    a = dict(q=FAKE, kp=FAKE, ks=None, vp=FAKE, vs=None, dtype=0, num_pages=100, kv_heads=2,
             table=FAKE, n_slots=4, max_pages=8, slots=FAKE, lens=FAKE, ids=FAKE, lists=2, topk=8,
             R=2, P=4, Hq=8, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, nb=1 << 30, stream=None)
    a.update(over)
    head = (a["q"], a["kp"], a["ks"], a["vp"], a["vs"], a["dtype"], a["num_pages"], a["kv_heads"],
            a["table"], a["n_slots"], a["max_pages"], a["slots"], a["lens"])
    tail = (a["R"], a["P"], a["Hq"], a["scale"], a["out"], a["lse"], a["ws"], a["nb"], a["stream"])
    if blocks:
        return L.idx_attn_blocks(*head, a["ids"], a["lists"], a["topk"], *tail)
    return L.idx_attn_paged(*head, *tail)


BAD = [
    (dict(R=-1), -1), (dict(R=2049), -1), (dict(P=0), -1), (dict(P=5000), -1), (dict(Hq=0), -1),
    (dict(Hq=7), -1), (dict(kv_heads=0), -1), (dict(kv_heads=3), -1), (dict(dtype=2), -2),
    (dict(dtype=7), -2), (dict(dtype=1), -1), (dict(dtype=1, ks=FAKE), -1), (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(n_slots=0), -1), (dict(max_pages=0), -1), (dict(max_pages=65537), -1),
    (dict(num_pages=0), -1), (dict(num_pages=1 << 24), -1), (dict(q=None), -1), (dict(kp=None), -1),
    (dict(vp=None), -1), (dict(table=None), -1), (dict(slots=None), -1), (dict(lens=None), -1),
    (dict(out=None), -1), (dict(ws=None), -1), (dict(ws=FAKE + 64), -1), (dict(nb=1000), -1),
    (dict(q=FAKE + 8), -1), (dict(kp=FAKE + 8), -1), (dict(vp=FAKE + 8), -1),
    (dict(dtype=1, ks=FAKE + 4, vs=FAKE), -1), (dict(R=2048, P=1, Hq=1024, kv_heads=1024), -1),
    (dict(table=FAKE + 2), -1), (dict(slots=FAKE + 1), -1), (dict(lens=FAKE + 2), -1), (dict(lse=FAKE + 2), -1),
]


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("over,status", BAD)
def test_attention_refusals(L, blocks, over, status):
    assert attn(L, blocks, **over) == status
    assert L.idx_last_error() != b""


@pytest.mark.parametrize("over", [dict(lists=0), dict(lists=-1), dict(lists=3), dict(topk=0),
                                  dict(topk=257), dict(ids=None), dict(Hq=12, lists=4, kv_heads=6),
                                  dict(lists=16)])
def test_block_attention_refusals(L, over):
    assert attn(L, True, **over) == -1
    assert L.idx_last_error() != b""


def test_workspace_bytes(L):
    assert idx.idx_attn_workspace_bytes(4, 16, 1) > 1024
    assert idx.idx_attn_workspace_bytes(4, 16, 1, 4) > 1024
    assert idx.idx_attn_workspace_bytes(0, 16, 1) == 0
    assert idx.idx_attn_workspace_bytes(4, 16, 3) == 0
    assert idx.idx_attn_workspace_bytes(4, 16, 2, 3) == 0
    assert idx.idx_attn_workspace_bytes(4, 16, 2, -1) == 0
    # the measured cases' and the example's scratch stays small
    assert max(idx.idx_attn_workspace_bytes(P, 16, 1, n) for P in (1, 4, 64) for n in (0, 1, 4)) < 64 << 20


def pool(dtype=0, pages=10, **over):
    p = _lib.IdxPool()
    p.dtype, p.page_size, p.dim, p.num_pages = dtype, 64, 128, pages
    p.payload = FAKE
    p.scale = FAKE if dtype else None
    p.payload_row_bytes = {0: 256, 1: 128, 2: 64}[dtype]
    p.scale_row_bytes = {0: 0, 1: 4, 2: 8}[dtype]
    for k, v in over.items():
        setattr(p, k, v)
    return p


def store(L, k=FAKE, v=FAKE, ks=256, vs=256, slots=FAKE, T=4, H=2, kp=None, vp=None):
    kp = pool() if kp is None else kp
    vp = pool() if vp is None else vp
    return L.idx_store_kv(k, v, ks, vs, slots, T, H, ctypes.byref(kp) if kp else None,
                          ctypes.byref(vp) if vp else None, None)


@pytest.mark.parametrize("over,status", [
    (dict(kp=False), -1), (dict(vp=False), -1), (dict(v=None), -1), (dict(H=0), -1), (dict(H=3), -1),
    (dict(T=-1), -1), (dict(T=1 << 40), -1), (dict(k=None), -1), (dict(slots=None), -1),
    (dict(ks=255), -1), (dict(ks=260), -1), (dict(vs=128), -1), (dict(k=FAKE + 2), -1),
    (dict(v=FAKE + 8), -1), (dict(kp=pool(2), vp=pool(2)), -2), (dict(kp=pool(1)), -1),
    (dict(vp=pool(1)), -1), (dict(vp=pool(pages=12)), -1), (dict(kp=pool(payload=None)), -1),
    (dict(kp=pool(1, scale=None), vp=pool(1)), -1), (dict(kp=pool(page_size=32)), -1),
    (dict(kp=pool(dim=64)), -1), (dict(kp=pool(payload_row_bytes=128)), -1),
    (dict(slots=FAKE + 4), -1), (dict(kp=pool(payload=FAKE + 8)), -1), (dict(kp=pool(1, scale=FAKE + 2), vp=pool(1)), -1),
])
def test_store_refusals(L, over, status):
    assert store(L, **over) == status
    assert L.idx_last_error() != b""


def test_store_of_nothing_is_a_no_op(L):
    assert store(L, T=0, k=None, v=FAKE, slots=None) == 0


def norm(L, **over):
    a = dict(x=FAKE, xs=256, r=FAKE, rs=256, w=FAKE, T=4, n=256, g=128, eps=1e-6, out=FAKE, sc=FAKE,
             res=FAKE)
    a.update(over)
    return L.idx_add_rmsnorm_fp8(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["T"], a["n"], a["g"],
                                 a["eps"], a["out"], a["sc"], a["res"], None)


@pytest.mark.parametrize("over", [
    dict(T=-1), dict(T=1 << 31), dict(n=0), dict(n=32769), dict(g=64), dict(g=-128), dict(eps=-1.0),
    dict(eps=float("nan")), dict(x=None), dict(w=None), dict(out=None), dict(sc=None), dict(xs=255),
    dict(rs=255), dict(x=FAKE + 1), dict(r=FAKE + 1), dict(w=FAKE + 1), dict(sc=FAKE + 2),
    dict(res=FAKE + 1), dict(rs=512)])
def test_norm_refusals(L, over):
    assert norm(L, **over) == -1
    assert L.idx_last_error() != b""


def test_norm_of_no_rows_is_a_no_op(L):
    assert norm(L, T=0, x=None, w=None) == 0


def test_cpu_tensors_and_wrong_shapes_are_refused():
    bf = torch.bfloat16
    x = torch.zeros((2, 128), dtype=bf)
    with pytest.raises(idx.IdxError):
        idx.idx_add_rmsnorm_fp8(x, None, x[0], 1e-6, 0, torch.zeros((2, 128), dtype=torch.uint8),
                                torch.zeros(2))
    with pytest.raises(idx.IdxError):
        idx.idx_store_kv(torch.zeros((1, 1, 128), dtype=bf), None, torch.zeros(1, dtype=torch.int64),
                         torch.zeros((64, 128), dtype=bf), None, None, None, "bf16", 1)
    q = torch.zeros((1, 1, 4, 128), dtype=bf)
    plane = torch.zeros((64, 128), dtype=bf)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(idx.IdxError):
        idx.idx_attn_paged(q, plane, None, plane, None, "bf16", i32(1, 1), i32(1), i32(1, 1), 1, 0.1,
                           q, None, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(idx.IdxError):
        idx.idx_attn_paged(q, plane, None, plane, None, "int3", i32(1, 1), i32(1), i32(1, 1), 1, 0.1,
                           q, None, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(idx.IdxError):
        idx.alloc_attn_workspace(1, 5, 2)
