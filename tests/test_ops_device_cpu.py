"""The four layer operators take tensors of the current device only, in both bindings (no GPU:
stand-ins with a tensor's attributes, and a library that refuses every call)."""
import pytest
import torch

import sparse_attention_indexer_packed_gb300 as idx
from sparse_attention_indexer_packed_gb300 import _lib

BF, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


class Stand:
    """What the bindings ask of a tensor."""

    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.device_index, self.is_cuda = dtype, torch.Size(shape), device, True
        self.real = torch.empty(shape, dtype=dtype, device="meta")
        self.nbytes = self.real.nbytes

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 0x10002          # misaligned: a library call that gets this far is refused

    def __getattr__(self, name):
        if name in ("stride", "is_contiguous", "element_size", "numel", "dim"):
            return getattr(self.real, name)
        raise AttributeError(name)


def calls():
    """Per operator: its arguments, tensors as stand-ins."""
    def cache(dtype):
        if dtype == "bf16":
            return [Stand(BF, 256, 128), None, Stand(BF, 256, 128), None]
        return [Stand(U8, 256, 128), Stand(F32, 256), Stand(U8, 256, 128), Stand(F32, 256)]

    def paged(dtype):
        return [Stand(BF, 2, 3, 4, 128), *cache(dtype), dtype, Stand(I32, 3, 5), Stand(I32, 2), Stand(I32, 2, 3)]

    tail = lambda: [2, 0.1, Stand(BF, 2, 3, 4, 128), Stand(F32, 2, 3, 4), Stand(U8, 1 << 24)]  # noqa: E731
    for dtype in ("bf16", "fp8_e4m3"):
        yield "idx_attn_paged", paged(dtype) + tail()
        yield "idx_attn_blocks", paged(dtype) + [Stand(I32, 2, 6, 7), 2] + tail()
        k, ks, v, vs = cache(dtype)
        yield "idx_store_kv", [Stand(BF, 9, 2, 128), Stand(BF, 9, 2, 128), Stand(I64, 9), k, ks, v, vs, dtype, 2]
    yield "idx_add_rmsnorm_fp8", [Stand(BF, 5, 300), Stand(BF, 5, 300), Stand(BF, 300), -1.0, 128,
                                  Stand(torch.float8_e4m3fn, 5, 300), Stand(F32, 5, 3), Stand(BF, 5, 300)]


CASES = list(calls())
NAMES = _lib.NATIVE_CALLS


@pytest.fixture
def bindings(monkeypatch):
    """{operator: call} of the Python functions and of the CPython module; current device 0."""
    import __graft_entry__
    __graft_entry__.build()
    from sparse_attention_indexer_packed_gb300 import _binding
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 0)
    python = {n: getattr(_lib, n) for n in NAMES}
    _binding.bind((BF, F32, I32, I64, U8, torch.float8_e4m3fn), lambda device: 0, lambda: 0, _lib._check,
                  tuple(python[n] for n in NAMES))
    yield python, {n: getattr(_binding, n) for n in NAMES}
    monkeypatch.undo()
    _lib._native_calls()       # the module's own objects again


@pytest.mark.parametrize("name,args", CASES)
def test_a_call_on_the_current_device_reaches_the_library(bindings, name, args):
    for fns in bindings:
        with pytest.raises(idx.IdxError, match="IDX_ERR_INVALID|invalid"):
            fns[name](*args)


@pytest.mark.parametrize("name,args", CASES)
def test_a_tensor_of_another_device_is_refused(bindings, name, args):
    tensors = [a for a in args if isinstance(a, Stand)]
    for group in [[t] for t in tensors] + [tensors]:
        for t in group:
            t.device_index = 1
        try:
            for fns in bindings:
                with pytest.raises(idx.IdxError, match="current device"):
                    fns[name](*args)
        finally:
            for t in group:
                t.device_index = 0


@pytest.mark.parametrize("name,args", CASES)
def test_a_stream_of_another_device_is_refused(bindings, name, args):
    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)

    for fns in bindings:
        with pytest.raises(idx.IdxError, match="current device"):
            fns[name](*args, stream=Stream())


def mutants(a):
    """Arguments like `a` and unlike it."""
    if isinstance(a, Stand):
        yield None
        yield 3
        for dtype in (BF, torch.float16, F32, I32, I64, U8):
            yield Stand(dtype, *a.shape)
        for d in range(len(a.shape)):
            yield Stand(a.dtype, *a.shape[:d], a.shape[d] + 1, *a.shape[d + 1:])
            yield Stand(a.dtype, *a.shape[:d], 0, *a.shape[d + 1:])
        yield Stand(a.dtype, *a.shape, 1)
        yield Stand(a.dtype, *a.shape[1:])
        apart = Stand(a.dtype, *a.shape)
        apart.real = torch.empty((2 * a.shape[0], *a.shape[1:]), dtype=a.dtype, device="meta")[::2]
        yield apart
        inner = Stand(a.dtype, *a.shape)
        inner.real = torch.empty((*a.shape, 2), dtype=a.dtype, device="meta")[..., 0]
        yield inner
        on_cpu = Stand(a.dtype, *a.shape, device=-1)
        on_cpu.is_cuda = False
        yield on_cpu
    else:
        yield from (None, 0, 1, 3, -1, 128, 0.5, -2.0, float("nan"), True, 1 << 40, "bf16", "fp8_e4m3", "nvfp4",
                    Stand(F32, 256))


@pytest.mark.parametrize("name,args", CASES)
def test_both_bindings_answer_alike(bindings, name, args):
    """What one accepts or refuses, and in which words, the other does too."""
    def answer(fn, a):
        try:
            return fn(*a)
        except Exception as e:  # noqa: BLE001 (any refusal)
            return type(e), str(e)

    python, module = bindings
    n = 0
    for at in range(len(args)):
        for m in mutants(args[at]):
            a = [*args[:at], m, *args[at + 1:]]
            assert answer(module[name], a) == answer(python[name], a), (at, m)
            n += 1
    assert n > 100
    for a in (args[:-1], args[:3], [], [*args, None]):
        assert answer(module[name], a) == answer(python[name], a)
