"""Host-side checks of the NVFP4 cache's operators and of the norm, rotation and store pass, in
the C ABI and in both bindings (no compute call runs)."""
import ctypes

import pytest
import torch

import sparse_attention_indexer_packed_gb300 as idx
from sparse_attention_indexer_packed_gb300 import _lib
from test_ops_abi_cpu import BAD, FAKE, pool
from test_ops_device_cpu import BF, F32, I32, I64, U8, Stand, bindings, mutants  # noqa: F401

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return idx.lib()


def attn(L, blocks=False, **over):
    a = dict(q=FAKE, kp=FAKE, ks=FAKE, vp=FAKE, vs=FAKE, num_pages=100, kv_heads=2, table=FAKE, n_slots=4,
             max_pages=8, slots=FAKE, lens=FAKE, ids=FAKE, lists=2, topk=8, R=2, P=4, Hq=8, scale=0.1, ko=1.0,
             vo=1.0, out=FAKE, lse=FAKE, ws=FAKE, nb=1 << 30, stream=None)
    a.update(over)
    head = (a["q"], a["kp"], a["ks"], a["vp"], a["vs"], a["num_pages"], a["kv_heads"], a["table"],
            a["n_slots"], a["max_pages"], a["slots"], a["lens"])
    tail = (a["R"], a["P"], a["Hq"], a["scale"], a["ko"], a["vo"], a["out"], a["lse"], a["ws"], a["nb"],
            a["stream"])
    if blocks:
        return L.idx_attn_blocks_nvfp4(*head, a["ids"], a["lists"], a["topk"], *tail)
    return L.idx_attn_paged_nvfp4(*head, *tail)


OUTERS = [0.0, -1.0, 3.0, 0.75, float("inf"), float("nan"), 2.0 ** -65, 2.0 ** 65, 1.0 + 2.0 ** -20]


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("over", [o for o, _ in BAD if "dtype" not in o]
                         + [dict(ks=None), dict(vs=None), dict(ks=FAKE + 8), dict(vs=FAKE + 4)]
                         + [{k: x} for k in ("ko", "vo") for x in OUTERS]
                         + [dict(scale=1e29, ko=2.0 ** 60), dict(scale=1e-30, ko=2.0 ** -60)])
def test_attention_refusals(L, blocks, over):
    assert attn(L, blocks, **over) == -1
    assert L.idx_last_error() != b""


@pytest.mark.parametrize("over", [dict(lists=0), dict(lists=3), dict(topk=0), dict(topk=257), dict(ids=None),
                                  dict(Hq=12, lists=4, kv_heads=6), dict(lists=16)])
def test_block_attention_refusals(L, over):
    assert attn(L, True, **over) == -1


def test_the_calls_of_the_other_types_still_refuse_nvfp4(L):
    p = pool(2)
    assert L.idx_store_kv(FAKE, None, 256, 0, FAKE, 4, 2, ctypes.byref(p), None, None) == -2
    assert L.idx_attn_paged(FAKE, FAKE, FAKE, FAKE, FAKE, 2, 100, 2, FAKE, 4, 8, FAKE, FAKE, 2, 4, 8, 0.1, FAKE,
                            None, FAKE, 1 << 30, None) == -2
    assert b"nvfp4" in L.idx_last_error()


def store(L, k=FAKE, v=FAKE, ks=256, vs=256, slots=FAKE, T=4, H=2, kp=None, vp=None, ko=1.0, vo=1.0):
    kp = pool(2) if kp is None else kp
    vp = pool(2) if vp is None else vp
    return L.idx_store_kv_nvfp4(k, v, ks, vs, slots, T, H, ctypes.byref(kp) if kp else None,
                                ctypes.byref(vp) if vp else None, ko, vo, None)


@pytest.mark.parametrize("over,status", [
    (dict(kp=False), -1), (dict(vp=False), -1), (dict(v=None), -1), (dict(H=0), -1), (dict(H=3), -1),
    (dict(T=-1), -1), (dict(T=1 << 40), -1), (dict(k=None), -1), (dict(slots=None), -1), (dict(ks=255), -1),
    (dict(vs=128), -1), (dict(k=FAKE + 2), -1), (dict(kp=pool(0), vp=pool(0)), -2), (dict(kp=pool(1)), -2),
    (dict(vp=pool(1)), -1), (dict(vp=pool(2, pages=12)), -1), (dict(kp=pool(2, scale=None)), -1),
    (dict(kp=pool(2, scale=FAKE + 4)), -1), (dict(kp=pool(2, payload=FAKE + 8)), -1),
    (dict(kp=pool(2, scale_row_bytes=4)), -1)] + [({k: x}, -1) for k in ("ko", "vo") for x in OUTERS])
def test_store_refusals(L, over, status):
    assert store(L, **over) == status
    assert L.idx_last_error() != b""


def test_a_store_of_nothing_is_a_no_op(L):
    assert store(L, T=0, k=None, v=None, slots=None) == 0
    # an empty tensor's pointer is NULL: not a source that was left out
    p = pool()
    assert L.idx_store_kv(None, None, 256, 256, None, 0, 2, ctypes.byref(p), ctypes.byref(p), None) == 0


def rope_of(**over):
    r = _lib.IdxRope()
    r.table, r.num_positions, r.positions, r.axes, r.rotary_dim = FAKE, 100, FAKE, 1, 128
    for k, v in over.items():
        if k == "pair_axis":
            r.pair_axis[v[0]] = v[1]
        else:
            setattr(r, k, v)
    return r


def norm_rope(L, **over):
    a = dict(q=FAKE, qs=512, Hq=4, k=FAKE, ks=512, v=FAKE, vs=512, H=2, qw=FAKE, kw=FAKE, eps=1e-6, rope=rope_of(),
             slots=FAKE, T=4, out=FAKE, outs=None, kp=pool(1), vp=pool(1), ko=1.0, vo=1.0)
    a.update(over)
    by = lambda x: ctypes.byref(x) if x else None  # noqa: E731
    return L.idx_norm_rope_store(a["q"], a["qs"], a["Hq"], a["k"], a["ks"], a["v"], a["vs"], a["H"], a["qw"], a["kw"],
                                 a["eps"], by(a["rope"]), a["slots"], a["T"], a["out"], a["outs"], by(a["kp"]),
                                 by(a["vp"]), a["ko"], a["vo"], None)


@pytest.mark.parametrize("over", [
    dict(q=None), dict(out=None), dict(q=None, out=None), dict(Hq=0), dict(Hq=-1), dict(Hq=32769, qs=1 << 24),
    dict(q=None, out=None, Hq=0, outs=FAKE), dict(k=None), dict(v=None), dict(vp=False), dict(kp=False), dict(H=0),
    dict(H=3), dict(slots=None), dict(T=-1), dict(T=1 << 34), dict(eps=-1.0), dict(eps=float("nan")), dict(qs=504),
    dict(ks=248), dict(vs=260), dict(q=FAKE + 8), dict(k=FAKE + 8), dict(v=FAKE + 8), dict(out=FAKE + 8),
    dict(qw=FAKE + 2), dict(kw=FAKE + 8), dict(slots=FAKE + 4), dict(outs=FAKE + 2), dict(kp=pool(1), vp=pool(2)),
    dict(kp=pool(1, scale=None)), dict(ko=2.0), dict(vo=0.5), dict(kp=pool(0), vp=pool(0), ko=2.0),
    dict(kp=pool(2), vp=pool(2), ko=3.0), dict(kp=pool(2), vp=pool(2, scale=FAKE + 4)),
] + [dict(rope=rope_of(**r)) for r in (
    dict(table=None), dict(positions=None), dict(table=FAKE + 8), dict(positions=FAKE + 2), dict(num_positions=0),
    dict(num_positions=1 << 31), dict(axes=0), dict(axes=5), dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=24),
    dict(rotary_dim=144), dict(axes=2, pair_axis=(5, 2)), dict(axes=3, pair_axis=(63, 3)))])
def test_norm_rope_refusals(L, over):
    assert norm_rope(L, **over) == -1
    assert L.idx_last_error() != b""


def test_no_tokens_is_a_no_op(L):
    assert norm_rope(L, T=0) == 0
    assert norm_rope(L, T=0, q=None, k=None, v=None, out=None, slots=None) == 0


# ---- the bindings ----------------------------------------------------------------------------
def calls():
    plane = lambda: [Stand(U8, 256, 64), Stand(U8, 256, 8), Stand(U8, 256, 64), Stand(E4M3, 256, 8)]  # noqa: E731
    head = [Stand(BF, 2, 3, 4, 128), *plane(), Stand(I32, 3, 5), Stand(I32, 2), Stand(I32, 2, 3)]
    tail = [2, 0.1, Stand(BF, 2, 3, 4, 128), Stand(F32, 2, 3, 4), Stand(U8, 1 << 24)]
    for outers in ([], [1.0, 0.5]):
        yield "idx_attn_paged_nvfp4", head + tail + outers
        yield "idx_attn_blocks_nvfp4", head + [Stand(I32, 2, 6, 7), 2] + tail + outers
        yield "idx_store_kv_nvfp4", [Stand(BF, 9, 2, 128), Stand(BF, 9, 2, 128), Stand(I64, 9), *plane(), 2] + outers
    for dtype in ("bf16", "fp8_e4m3", "nvfp4"):
        cache = {"bf16": [Stand(BF, 256, 128), None] * 2, "nvfp4": plane(),
                 "fp8_e4m3": [Stand(U8, 256, 128), Stand(F32, 256)] * 2}[dtype]
        yield "idx_norm_rope_store", [
            Stand(BF, 9, 4, 128), Stand(BF, 9, 2, 128), Stand(BF, 9, 2, 128), Stand(BF, 128), Stand(BF, 128), 1e-6,
            Stand(F32, 50, 32), Stand(I32, 2, 9), bytes(i % 2 for i in range(16)), False, Stand(I64, 9),
            Stand(BF, 9, 4, 128), None, *cache, dtype, 2]
    yield "idx_norm_rope_store", [
        Stand(BF, 9, 4, 128), Stand(BF, 9, 2, 128), None, None, Stand(BF, 128), 1e-6, Stand(F32, 50, 32), Stand(I32, 9),
        None, True, Stand(I64, 9), Stand(E4M3, 9, 4, 128), Stand(F32, 9, 4), *plane()[:2], None, None, "nvfp4", 2, 2.0, 1.0]
    yield "idx_norm_rope_store", [
        None, Stand(BF, 9, 2, 128), Stand(BF, 9, 2, 128), None, None, 0.0, None, None, None, False, Stand(I64, 9), None,
        None, *plane(), "nvfp4", 2]


CASES = list(calls())


@pytest.mark.parametrize("name,args", CASES)
def test_a_call_on_the_current_device_reaches_the_library(bindings, name, args):  # noqa: F811
    for fns in bindings:
        with pytest.raises(idx.IdxError, match="IDX_ERR_INVALID"):
            fns[name](*args)


@pytest.mark.parametrize("name,args", CASES)
def test_a_tensor_of_another_device_is_refused(bindings, name, args):  # noqa: F811
    for t in [a for a in args if isinstance(a, Stand)]:
        t.device_index = 1
        try:
            for fns in bindings:
                with pytest.raises(idx.IdxError, match="current device"):
                    fns[name](*args)
        finally:
            t.device_index = 0


@pytest.mark.parametrize("name,args", CASES)
def test_both_bindings_answer_alike(bindings, name, args):  # noqa: F811
    def answer(fn, a):
        try:
            return fn(*a)
        except Exception as e:  # noqa: BLE001 (any refusal)
            return type(e), str(e)

    python, module = bindings
    n = 0
    for at in range(len(args)):
        more = (b"\0" * 16, b"\0" * 15, b"", b"\1" * 16, b"\2" * 16) if name == "idx_norm_rope_store" and at == 8 else ()
        for m in [*mutants(args[at]), *more]:
            a = [*args[:at], m, *args[at + 1:]]
            assert answer(module[name], a) == answer(python[name], a), (at, m)
            n += 1
    assert n > 80
    for a in (args[:-1], args[:3], [], [*args, None], [*args, 1.0, 2.0]):
        assert answer(module[name], a) == answer(python[name], a)


def test_cpu_tensors_and_wrong_planes_are_refused():
    x = torch.zeros((1, 1, 128), dtype=BF)
    slots = torch.zeros(1, dtype=I64)
    plane = torch.zeros((64, 64), dtype=U8)
    for scale in (None, torch.zeros((64, 8), dtype=U8), torch.zeros((64, 2)), torch.zeros((64, 4), dtype=U8)):
        with pytest.raises(idx.IdxError):
            idx.idx_store_kv_nvfp4(x, None, slots, plane, scale, None, None, 1)
    with pytest.raises(idx.IdxError):
        idx.idx_norm_rope_store(None, x, None, None, None, 0.0, None, None, None, False, slots, None, None,
                                torch.zeros((64, 128), dtype=BF), None, None, None, "bf16", 1)
