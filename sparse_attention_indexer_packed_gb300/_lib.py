"""ctypes binding of libidx (include/idx.h): argument marshalling only.

Every function here forwards to the C ABI of the same name with the device
pointers of the torch tensors it is given; all arithmetic runs in the library's
CUDA kernels.  There is no CPU path: a tensor that is not on a CUDA device, or a
missing libidx.so, raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libidx.so")

IDX_BF16, IDX_FP8_E4M3, IDX_NVFP4 = 0, 1, 2
IDX_OK = 0
PAGE, BLOCK, DIM = 64, 128, 128
WORKSPACE_HEADER_BYTES = 1024
DEVERR_BAD_PAGE, DEVERR_TIMEOUT, DEVERR_LEN_CLAMPED = 1, 2, 4

DTYPES = {"bf16": IDX_BF16, "fp8_e4m3": IDX_FP8_E4M3, "nvfp4": IDX_NVFP4}


class IdxPool(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("payload", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("payload_row_bytes", ctypes.c_int64),
                ("scale_row_bytes", ctypes.c_int64)]


class IdxError(RuntimeError):
    pass


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float

_SIGNATURES = {
    "idx_abi_version": (_I, []),
    "idx_status_string": (ctypes.c_char_p, [_I]),
    "idx_last_error": (ctypes.c_char_p, []),
    "idx_pool_alloc": (_I, [_I, _I64, _I, _I, ctypes.POINTER(IdxPool)]),
    "idx_pool_free": (_I, [ctypes.POINTER(IdxPool)]),
    "idx_store_nvfp4": (_I, [_P, _P, _I64, ctypes.POINTER(IdxPool), _P]),
    "idx_score_topk_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "idx_score_topk": (_I, [_P, _P, _I, _P, _P, _I, _I64, _P, _I, _I, _P, _P, _I, _I, _I,
                            _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "idx_score_topk_lse": (_I, [_P, _P, _I, _P, _P, _I, _I64, _P, _I, _I, _P, _P, _I, _I, _I,
                                _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "idx_score_topk_perrow": (_I, [_P, _P, _I, _P, _P, _I, _I64, _P, _I, _I, _P, _P, _I, _I,
                                   _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "idx_score_local_blocks": (_I, [_P, _P, _I, _P, _P, _I, _I64, _P, _I, _I, _I, _P, _P, _I,
                                    _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "idx_set_wait_limit_ns": (_I, [ctypes.c_uint64]),
    "idx_set_stall_test": (_I, [_I]),
    "idx_topk_merge": (_I, [_P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "idx_score_topk_noalloc": (_I, [_P, _P, _I, _P, _P, _I, _I64, _P, _I, _I, _P, _P, _I, _I,
                                    _I, _I, _I, _I, _P, _P, _P]),
    # (the pools are passed as the struct's bytes: see _pool_bytes)
    "idx_store_kv": (_I, [_P, _P, _I64, _I64, _P, _I64, _I, _P, _P, _P]),
    "idx_attn_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "idx_attn_paged": (_I, [_P, _P, _P, _P, _P, _I, _I64, _I, _P, _I, _I, _P, _P, _I, _I, _I, _F,
                            _P, _P, _P, _SZ, _P]),
    "idx_attn_blocks": (_I, [_P, _P, _P, _P, _P, _I, _I64, _I, _P, _I, _I, _P, _P, _P, _I, _I, _I,
                             _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "idx_store_kv_nvfp4": (_I, [_P, _P, _I64, _I64, _P, _I64, _I, _P, _P, _F, _F, _P]),
    "idx_attn_paged_nvfp4": (_I, [_P, _P, _P, _P, _P, _I64, _I, _P, _I, _I, _P, _P, _I, _I, _I, _F, _F,
                                  _F, _P, _P, _P, _SZ, _P]),
    "idx_attn_blocks_nvfp4": (_I, [_P, _P, _P, _P, _P, _I64, _I, _P, _I, _I, _P, _P, _P, _I, _I, _I,
                                   _I, _I, _F, _F, _F, _P, _P, _P, _SZ, _P]),
    # (the rotation is passed as the struct's bytes: see _rope_bytes)
    "idx_norm_rope_store": (_I, [_P, _I64, _I, _P, _I64, _P, _I64, _I, _P, _P, _F, _P, _P, _I64, _P, _P,
                                 _P, _P, _F, _F, _P]),
    "idx_add_rmsnorm_fp8": (_I, [_P, _I64, _P, _I64, _P, _I64, _I, _I, _F, _P, _P, _P, _P]),
    "idx_set_kernel_events": (_I, [_P, _P, _P]),
    "idx_set_kernel_waits": (_I, [_P, _P]),
    "idx_set_grid_limit": (_I, [_I]),
    "idx_workspace_errors": (_I, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "idx_noalloc_errors": (_I, [_P, ctypes.POINTER(ctypes.c_uint32)]),
}


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise IdxError(f"{LIB_PATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(rc: int, what: str) -> None:
    if rc != IDX_OK:
        msg = lib().idx_last_error().decode()
        name = lib().idx_status_string(rc).decode()
        raise IdxError(f"{what} failed: {name}: {msg}")


def _dev(t: Optional[torch.Tensor], name: str, required: bool = True) -> Optional[int]:
    if t is None:
        if required:
            raise IdxError(f"{name} is required")
        return None
    if not t.is_cuda:
        raise IdxError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise IdxError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# torch.cuda.current_stream() builds a Stream object (~3 us); a decode step's small
# calls ask torch for the bare handle where it has that call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(t: torch.Tensor, stream) -> Optional[int]:
    """The given stream's handle, or that of t's device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _raw_stream(t.get_device())


def _one_device(stream, *tensors) -> None:
    """The library launches on the current device: everything has to be there (CUDA tensors,
    None where an argument is left out)."""
    here = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise IdxError(f"a tensor is on cuda:{t.get_device()} and the current device is cuda:{here}: "
                           "all of a call's tensors must be on the current device (torch.cuda.device)")
    if stream is not None and stream.device.index != here:
        raise IdxError(f"the stream is of {stream.device} and the current device is cuda:{here}")


def pool_struct(dtype: str, payload: torch.Tensor, scale: Optional[torch.Tensor]) -> IdxPool:
    """Describe caller-owned planes (torch tensors) as an idx_pool."""
    rows, row_bytes = payload.shape[0], payload.shape[1] * payload.element_size()
    p = IdxPool()
    p.dtype = DTYPES[dtype]
    p.page_size = PAGE
    p.dim = DIM
    p.num_pages = rows // PAGE
    p.payload = _dev(payload, "payload")
    p.scale = _dev(scale, "scale", required=False)
    p.payload_row_bytes = row_bytes
    p.scale_row_bytes = 0 if scale is None else scale.shape[1] * scale.element_size()
    return p


def abi_version() -> int:
    return lib().idx_abi_version()


def idx_pool_alloc(dtype: str, num_pages: int) -> IdxPool:
    p = IdxPool()
    _check(lib().idx_pool_alloc(DTYPES[dtype], num_pages, PAGE, DIM, ctypes.byref(p)),
           "idx_pool_alloc")
    return p


def idx_pool_free(pool: IdxPool) -> None:
    _check(lib().idx_pool_free(ctypes.byref(pool)), "idx_pool_free")


def idx_store_nvfp4(src_bf16: torch.Tensor, slot_mapping: torch.Tensor, pool, stream=None) -> None:
    """pool: an IdxPool, or a (payload, scale) pair of uint8 tensors."""
    if isinstance(pool, tuple):
        pool = pool_struct("nvfp4", pool[0], pool[1])
    if src_bf16.dtype != torch.bfloat16 or slot_mapping.dtype != torch.int64:
        raise IdxError("src_bf16 must be bfloat16 and slot_mapping int64")
    n = int(slot_mapping.numel())
    _check(lib().idx_store_nvfp4(_dev(src_bf16, "src_bf16"), _dev(slot_mapping, "slot_mapping"),
                                 n, ctypes.byref(pool), _stream_ptr(stream)), "idx_store_nvfp4")


def idx_score_topk_workspace_bytes(num_requests: int, packed_queries: int, gqa: int,
                                   max_pages: int) -> int:
    return int(lib().idx_score_topk_workspace_bytes(num_requests, packed_queries, gqa, max_pages))


def alloc_workspace(num_requests: int, packed_queries: int, gqa: int, max_pages: int,
                    device="cuda") -> torch.Tensor:
    n = idx_score_topk_workspace_bytes(num_requests, packed_queries, gqa, max_pages)
    return torch.empty(max(n, WORKSPACE_HEADER_BYTES), dtype=torch.uint8, device=device)


def _q_dtype(q: torch.Tensor) -> int:
    if q.dtype == torch.bfloat16:
        return IDX_BF16
    if q.dtype in (torch.uint8, torch.float8_e4m3fn):
        return IDX_FP8_E4M3
    raise IdxError(f"unsupported q dtype {q.dtype}")


def _score(fn_name: str, q, q_scale, k_payload, k_scale, k_dtype: str, page_table, slot_ids,
           row_lens, packed_queries, gqa, init_blocks, local_blocks, topk, out_ids, out_scores,
           workspace, stream):
    R = int(q.shape[0])
    num_pages = int(k_payload.shape[0]) // PAGE
    n_slots, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    for t, name, dt in [(page_table, "page_table", torch.int32), (slot_ids, "slot_ids", torch.int32),
                        (row_lens, "row_lens", torch.int32), (out_ids, "out_ids", torch.int32),
                        (out_scores, "out_scores", torch.float32)]:
        if t.dtype != dt:
            raise IdxError(f"{name} must be {dt}")
    fn = getattr(lib(), fn_name)
    rc = fn(_dev(q, "q"), _dev(q_scale, "q_scale", required=False), _q_dtype(q),
            _dev(k_payload, "k_payload"), _dev(k_scale, "k_scale", required=False),
            DTYPES[k_dtype], num_pages, _dev(page_table, "page_table"), n_slots, max_pages,
            _dev(slot_ids, "slot_ids"), _dev(row_lens, "row_lens"), R, packed_queries, gqa,
            init_blocks, local_blocks, topk, _dev(out_ids, "out_ids"),
            _dev(out_scores, "out_scores"), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check(rc, fn_name)


def idx_score_topk(q, q_scale, k_payload, k_scale, k_dtype, page_table, slot_ids, row_lens,
                   packed_queries, gqa, init_blocks, local_blocks, topk, out_ids, out_scores,
                   workspace, stream=None) -> None:
    _score("idx_score_topk", q, q_scale, k_payload, k_scale, k_dtype, page_table, slot_ids,
           row_lens, packed_queries, gqa, init_blocks, local_blocks, topk, out_ids, out_scores,
           workspace, stream)


def idx_score_topk_lse(q, q_scale, k_payload, k_scale, k_dtype, page_table, slot_ids, row_lens,
                       packed_queries, gqa, init_blocks, local_blocks, topk, out_ids, out_scores,
                       workspace, stream=None) -> None:
    _score("idx_score_topk_lse", q, q_scale, k_payload, k_scale, k_dtype, page_table, slot_ids,
           row_lens, packed_queries, gqa, init_blocks, local_blocks, topk, out_ids, out_scores,
           workspace, stream)


def idx_score_topk_perrow(q, q_scale, k_payload, k_scale, k_dtype, page_table, slot_ids, row_lens,
                          packed_queries, gqa, init_blocks, local_blocks, topk, out_ids,
                          out_scores, workspace, stream=None) -> None:
    _score("idx_score_topk_perrow", q, q_scale, k_payload, k_scale, k_dtype, page_table, slot_ids,
           row_lens, packed_queries, gqa, init_blocks, local_blocks, topk, out_ids, out_scores,
           workspace, stream)


def idx_score_local_blocks(q, q_scale, k_payload, k_scale, k_dtype, page_table, block_begin,
                           slot_ids, row_lens, packed_queries, gqa, init_blocks, local_blocks,
                           topk, out_ids, out_scores, workspace, stream=None) -> None:
    """One context shard: page_table [n_slots, max_pages] covers global blocks
    [block_begin, block_begin + max_pages / 2) of every request."""
    R = int(q.shape[0])
    num_pages = int(k_payload.shape[0]) // PAGE
    n_slots, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    for t, name, dt in [(page_table, "page_table", torch.int32), (slot_ids, "slot_ids", torch.int32),
                        (row_lens, "row_lens", torch.int32), (out_ids, "out_ids", torch.int32),
                        (out_scores, "out_scores", torch.float32)]:
        if t.dtype != dt:
            raise IdxError(f"{name} must be {dt}")
    rc = lib().idx_score_local_blocks(
        _dev(q, "q"), _dev(q_scale, "q_scale", required=False), _q_dtype(q),
        _dev(k_payload, "k_payload"), _dev(k_scale, "k_scale", required=False), DTYPES[k_dtype],
        num_pages, _dev(page_table, "page_table"), n_slots, max_pages, int(block_begin),
        _dev(slot_ids, "slot_ids"), _dev(row_lens, "row_lens"), R, packed_queries, gqa,
        init_blocks, local_blocks, topk, _dev(out_ids, "out_ids"), _dev(out_scores, "out_scores"),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(rc, "idx_score_local_blocks")


def idx_topk_merge(cand_ids, cand_scores, slot_ids, row_lens, n_slots, packed_queries, gqa,
                   init_blocks, local_blocks, topk, out_ids, out_scores, stream=None) -> None:
    """cand_ids / cand_scores: [world, R, P*G, topk], the shards' lists."""
    world, R = int(cand_ids.shape[0]), int(cand_ids.shape[1])
    for t, name, dt in [(cand_ids, "cand_ids", torch.int32), (cand_scores, "cand_scores", torch.float32),
                        (slot_ids, "slot_ids", torch.int32), (row_lens, "row_lens", torch.int32),
                        (out_ids, "out_ids", torch.int32), (out_scores, "out_scores", torch.float32)]:
        if t.dtype != dt:
            raise IdxError(f"{name} must be {dt}")
    rc = lib().idx_topk_merge(_dev(cand_ids, "cand_ids"), _dev(cand_scores, "cand_scores"), world,
                              _dev(slot_ids, "slot_ids"), _dev(row_lens, "row_lens"), int(n_slots),
                              R, packed_queries, gqa, init_blocks, local_blocks, topk,
                              _dev(out_ids, "out_ids"), _dev(out_scores, "out_scores"),
                              _stream_ptr(stream))
    _check(rc, "idx_topk_merge")


def idx_set_wait_limit_ns(ns: int) -> None:
    """Limit of the score kernels' pipeline waits (0: the default 2 s)."""
    _check(lib().idx_set_wait_limit_ns(int(ns)), "idx_set_wait_limit_ns")


def idx_set_stall_test(on: bool) -> None:
    """Diagnostic: one role per score CTA waits on a barrier nothing completes."""
    _check(lib().idx_set_stall_test(1 if on else 0), "idx_set_stall_test")


def idx_set_kernel_events(score_begin=None, score_end=None, topk_end=None) -> None:
    """Arm torch.cuda.Event objects (enable_timing=True) for the next score call."""
    h = [None if e is None else e.cuda_event for e in (score_begin, score_end, topk_end)]
    _check(lib().idx_set_kernel_events(*h), "idx_set_kernel_events")


def idx_set_kernel_waits(before_score=None, before_topk=None) -> None:
    """Arm torch.cuda.Event objects the next score call's stream waits for before
    its score kernel / its top-k kernel (include/idx.h: idx_set_kernel_waits)."""
    h = [None if e is None else e.cuda_event for e in (before_score, before_topk)]
    _check(lib().idx_set_kernel_waits(*h), "idx_set_kernel_waits")


def idx_score_topk_noalloc(q, q_scale, k_payload, k_scale, k_dtype, page_table, slot_ids,
                           row_lens, packed_queries, gqa, init_blocks, local_blocks, topk,
                           out_ids, out_scores, stream=None) -> None:
    """idx_score_topk with the library's fixed scratch array instead of a workspace,
    for callers that cannot allocate device memory (see include/idx.h)."""
    R = int(q.shape[0])
    n_slots, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
    rc = lib().idx_score_topk_noalloc(
        _dev(q, "q"), _dev(q_scale, "q_scale", required=False), _q_dtype(q),
        _dev(k_payload, "k_payload"), _dev(k_scale, "k_scale", required=False), DTYPES[k_dtype],
        int(k_payload.shape[0]) // PAGE, _dev(page_table, "page_table"), n_slots, max_pages,
        _dev(slot_ids, "slot_ids"), _dev(row_lens, "row_lens"), R, packed_queries, gqa,
        init_blocks, local_blocks, topk, _dev(out_ids, "out_ids"), _dev(out_scores, "out_scores"),
        _stream_ptr(stream))
    _check(rc, "idx_score_topk_noalloc")


def idx_set_grid_limit(max_ctas: int) -> None:
    """Cap the score kernel's grid (0 = one CTA per SM); results do not change."""
    _check(lib().idx_set_grid_limit(int(max_ctas)), "idx_set_grid_limit")


def idx_workspace_errors(workspace: torch.Tensor, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(lib().idx_workspace_errors(_dev(workspace, "workspace"), _stream_ptr(stream),
                                      ctypes.byref(v)), "idx_workspace_errors")
    return int(v.value)


def idx_noalloc_errors(stream=None) -> int:
    """Device error flags of the last idx_score_topk_noalloc call on this device."""
    v = ctypes.c_uint32(0)
    _check(lib().idx_noalloc_errors(_stream_ptr(stream), ctypes.byref(v)), "idx_noalloc_errors")
    return int(v.value)


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_ROW_BYTES = {"bf16": 256, "fp8_e4m3": 128, "nvfp4": 64}
_SCALE_BYTES = {"bf16": 0, "fp8_e4m3": 4, "nvfp4": 8}


def _want(t: torch.Tensor, name: str, dtype, shape) -> int:
    """Device pointer of a contiguous CUDA tensor of this dtype and shape."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise IdxError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise IdxError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return _dev(t, name)


def _rows_2d(t: torch.Tensor, name: str, rows: int, width: int):
    """Device pointer and row stride of a bf16 tensor whose rows are contiguous."""
    if t.dtype is not _BF16 or t.shape != (rows, width):
        raise IdxError(f"{name} must be bfloat16 [{rows}, {width}]")
    if not t.is_cuda:
        raise IdxError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    stride, inner = t.stride()
    if width > 1 and inner != 1:
        raise IdxError(f"{name}'s rows must be contiguous")
    return t.data_ptr(), (stride if rows > 1 else width)


def _plane(payload, scale, name: str, kv_dtype: str):
    """Pointers of a plane and its head pages, checked against the cache's dtype."""
    want = _ROW_BYTES.get(kv_dtype)
    if want is None:
        raise IdxError(f"unknown dtype {kv_dtype!r}")
    shape = payload.shape
    if len(shape) != 2 or shape[1] * payload.element_size() != want:
        raise IdxError(f"{name}_payload must be [rows, {want} bytes] for a {kv_dtype} cache")
    rows = shape[0]
    if rows % PAGE:
        raise IdxError(f"{name}_payload must hold whole pages of {PAGE} rows")
    if scale is not None or kv_dtype == "fp8_e4m3":
        if kv_dtype == "fp8_e4m3" and (scale is None or scale.nbytes != rows * 4):
            raise IdxError(f"{name}_scale must hold one fp32 per row")
        scale = _dev(scale, f"{name}_scale")
    return _dev(payload, f"{name}_payload"), scale, rows // PAGE


def _plane4(payload, scale, name: str):
    """_plane of an NVFP4 cache, whose scales are required."""
    ptr, _, pages = _plane(payload, None, name, "nvfp4")
    if (scale is None or scale.dtype not in (torch.uint8, torch.float8_e4m3fn)
            or scale.shape != (pages * PAGE, DIM // 16)):
        raise IdxError(f"{name}_scale must be uint8 or float8_e4m3fn [{pages * PAGE}, {DIM // 16}]")
    return ptr, _dev(scale, f"{name}_scale"), pages


def _source(src, name: str, tokens: int, kv_heads: int):
    """Pointer and token stride of new keys or values [tokens, kv_heads, 128]."""
    if src.dtype is not _BF16 or src.shape != (tokens, kv_heads, DIM):
        raise IdxError(f"{name} must be bfloat16 [{tokens}, {kv_heads}, {DIM}]")
    if not src.is_cuda:
        raise IdxError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    stride, head, inner = src.stride()
    if tokens and (inner != 1 or (kv_heads > 1 and head != DIM)):
        raise IdxError(f"{name}'s tokens must be contiguous [{kv_heads}, {DIM}]")
    return src.data_ptr(), (stride if tokens > 1 else kv_heads * DIM)


# IdxPool's fields (checked below): packing them is a tenth of filling a ctypes struct.
_POOL = struct.Struct("=iiiiqQQqq")
assert _POOL.size == ctypes.sizeof(IdxPool)


def _pool_bytes(payload, scale, name: str, kv_dtype: str) -> bytes:
    ptr, scale_ptr, pages = (_plane4(payload, scale, name) if kv_dtype == "nvfp4" else
                             _plane(payload, scale, name, kv_dtype))
    return _POOL.pack(DTYPES[kv_dtype], PAGE, DIM, 0, pages, ptr, scale_ptr or 0,
                      _ROW_BYTES[kv_dtype], _SCALE_BYTES[kv_dtype])


def _store_args(k_src, v_src, slot_mapping, k_payload, k_scale, v_payload, v_scale, kv_dtype, kv_heads, stream):
    """The arguments the two store calls begin with."""
    if k_src is None or k_payload is None or (v_src is None) != (v_payload is None):
        raise IdxError("a source and its payload plane come together, and the keys always")
    T = slot_mapping.numel()
    k_ptr, k_stride = _source(k_src, "k_src", T, kv_heads)
    k_pool = _pool_bytes(k_payload, k_scale, "k", kv_dtype)
    v_ptr, v_stride, v_pool = None, 0, None
    if v_src is not None:
        v_ptr, v_stride = _source(v_src, "v_src", T, kv_heads)
        v_pool = _pool_bytes(v_payload, v_scale, "v", kv_dtype)
    slots = _want(slot_mapping, "slot_mapping", torch.int64, (T,))
    _one_device(stream, k_src, v_src, slot_mapping, k_payload, k_scale, v_payload, v_scale)
    return k_ptr, v_ptr, k_stride, v_stride, slots, T, kv_heads, k_pool, v_pool


def idx_store_kv(k_src, v_src, slot_mapping, k_payload, k_scale, v_payload, v_scale,
                 kv_dtype: str, kv_heads: int, stream=None) -> None:
    """k_src, v_src: bf16 [tokens, kv_heads, 128], tokens any stride apart (a slice of a
    fused projection); v_src, v_payload, v_scale None: keys only.  slot_mapping: int64, page *
    64 + offset, every token's its own (negative: skipped).  Planes as for idx_attn_paged, or
    an index pool's (kv_heads 1)."""
    args = _store_args(k_src, v_src, slot_mapping, k_payload, k_scale, v_payload, v_scale, kv_dtype,
                       kv_heads, stream)
    rc = lib().idx_store_kv(*args, _stream_of(k_src, stream))
    if rc:
        _check(rc, "idx_store_kv")


def idx_store_kv_nvfp4(k_src, v_src, slot_mapping, k_payload, k_scale, v_payload, v_scale,
                       kv_heads: int, k_outer: float = 1.0, v_outer: float = 1.0, stream=None) -> None:
    """idx_store_kv into NVFP4 planes: payload [rows, 64] bytes, scale uint8 (or float8_e4m3fn)
    [rows, 8]; value = code * scale * outer, outer a power of two for each plane."""
    args = _store_args(k_src, v_src, slot_mapping, k_payload, k_scale, v_payload, v_scale, "nvfp4",
                       kv_heads, stream)
    rc = lib().idx_store_kv_nvfp4(*args, k_outer, v_outer, _stream_of(k_src, stream))
    if rc:
        _check(rc, "idx_store_kv_nvfp4")


class IdxRope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("num_positions", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("axes", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("pair_axis", ctypes.c_uint8 * 64)]


_ROPE = struct.Struct("=QqQiiii64s")
assert _ROPE.size == ctypes.sizeof(IdxRope)


def _rope_bytes(table, positions, pair_axis, interleaved, tokens: int):
    """The rotation as the struct's bytes; None without a table."""
    if table is None:
        if positions is not None or pair_axis is not None:
            raise IdxError("positions and pair_axis come with a table")
        return None
    if table.dim() != 2 or positions is None:
        raise IdxError("table must be [num_positions, rotary_dim], and positions go with it")
    axes = positions.shape[0] if positions.dim() == 2 else 1
    shape = (axes, tokens) if positions.dim() == 2 else (tokens,)
    by = b"" if pair_axis is None else bytes(pair_axis)
    if (axes > 1 or by) and len(by) != table.shape[1] // 2:
        raise IdxError(f"pair_axis must name an axis for each of the {table.shape[1] // 2} pairs (got {len(by)})")
    if len(by) > 64:
        raise IdxError("rotary_dim must be at most 128")
    return _ROPE.pack(_want(table, "table", _F32, table.shape), table.shape[0],
                      _want(positions, "positions", _I32, shape), axes, table.shape[1],
                      bool(interleaved), 0, by)


def idx_norm_rope_store(q, k, v, q_weight, k_weight, eps: float, table, positions, pair_axis, interleaved: bool,
                        slot_mapping, out_q, out_q_scale, k_payload, k_scale, v_payload, v_scale,
                        kv_dtype: str, kv_heads: int, k_outer: float = 1.0, v_outer: float = 1.0,
                        stream=None) -> None:
    """Norm, rotation and store of a projection's parts.  q [tokens, q_heads, 128] (or None), k and
    v (or None) [tokens, kv_heads, 128]: bf16, tokens any stride apart.  q_weight, k_weight: bf16
    [128], or None: no norm.  table: fp32 [num_positions, rotary_dim], cosines then sines, or None: no
    rotation; positions: int32 [tokens] or [axes, tokens]; pair_axis: the axis of each pair (bytes,
    rotary_dim / 2 of them; None with one axis).  out_q [tokens, q_heads, 128]: bf16, or e4m3 codes with
    out_q_scale fp32 [tokens, q_heads].  Planes as for the store calls."""
    if k is None or k_payload is None or (v is None) != (v_payload is None) or (q is None) != (out_q is None):
        raise IdxError("k and its plane are required, v and its plane, q and out_q come together")
    T = slot_mapping.numel()
    qp, qs, Hq, outq, outs = None, 0, 0, None, None
    if q is not None:
        if q.dim() != 3:
            raise IdxError(f"q must be [tokens, q_heads, {DIM}]")
        Hq = q.shape[1]
        qp, qs = _source(q, "q", T, Hq)
        if out_q_scale is None:
            outq = _want(out_q, "out_q", _BF16, q.shape)
        else:
            if out_q.dtype is not torch.float8_e4m3fn and out_q.dtype is not torch.uint8:
                raise IdxError("out_q must be float8_e4m3fn or uint8 with out_q_scale")
            outq = _want(out_q, "out_q", out_q.dtype, q.shape)
            outs = _want(out_q_scale, "out_q_scale", _F32, (T, Hq))
    elif out_q_scale is not None:
        raise IdxError("out_q_scale comes with q")
    kp, ks = _source(k, "k", T, kv_heads)
    k_pool = _pool_bytes(k_payload, k_scale, "k", kv_dtype)
    vp, vs, v_pool = None, 0, None
    if v is not None:
        vp, vs = _source(v, "v", T, kv_heads)
        v_pool = _pool_bytes(v_payload, v_scale, "v", kv_dtype)
    weights = [None if w is None else _want(w, n, _BF16, (DIM,))
               for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight"))]
    rope = _rope_bytes(table, positions, pair_axis, interleaved, T)
    slots = _want(slot_mapping, "slot_mapping", torch.int64, (T,))
    _one_device(stream, q, k, v, q_weight, k_weight, table, positions, slot_mapping, out_q, out_q_scale,
                k_payload, k_scale, v_payload, v_scale)
    rc = lib().idx_norm_rope_store(qp, qs, Hq, kp, ks, vp, vs, kv_heads, *weights, eps, rope, slots, T, outq,
                                   outs, k_pool, v_pool, k_outer, v_outer, _stream_of(k, stream))
    if rc:
        _check(rc, "idx_norm_rope_store")


def idx_attn_workspace_bytes(packed_queries: int, q_heads: int, kv_heads: int, lists: int = 0) -> int:
    return int(lib().idx_attn_workspace_bytes(packed_queries, q_heads, kv_heads, lists))


def alloc_attn_workspace(packed_queries: int, q_heads: int, kv_heads: int, lists: int = 0,
                         device="cuda") -> torch.Tensor:
    n = idx_attn_workspace_bytes(packed_queries, q_heads, kv_heads, lists)
    if n == 0:
        raise IdxError(f"no attention of {packed_queries} draft rows, {q_heads} query heads, "
                       f"{kv_heads} key heads and {lists} lists")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _attn_args(q, k_payload, k_scale, v_payload, v_scale, kv_dtype, page_table, slot_ids,
               row_lens, kv_heads):
    """The arguments the two attention calls begin with, and R, P, q_heads."""
    shape = q.shape
    if len(shape) != 4 or shape[3] != DIM:
        raise IdxError(f"q must be [requests, draft rows, q_heads, {DIM}]")
    R, P, Hq, _ = shape
    if kv_dtype is None:   # NVFP4: the call's name says so
        (kp, ks, k_pages), (vp, vs, v_pages) = _plane4(k_payload, k_scale, "k"), _plane4(v_payload, v_scale, "v")
    else:
        kp, ks, k_pages = _plane(k_payload, k_scale, "k", kv_dtype)
        vp, vs, v_pages = _plane(v_payload, v_scale, "v", kv_dtype)
    if kv_heads < 1 or k_pages != v_pages or k_pages % kv_heads:
        raise IdxError("the planes must hold the same whole pages of kv_heads heads")
    table = page_table.shape
    if len(table) != 2:
        raise IdxError("page_table must be [n_slots, max_pages]")
    n_slots, max_pages = table
    return (_want(q, "q", _BF16, shape), kp, ks, vp, vs,
            *(() if kv_dtype is None else (DTYPES[kv_dtype],)), k_pages // kv_heads, kv_heads,
            _want(page_table, "page_table", _I32, table), n_slots, max_pages,
            _want(slot_ids, "slot_ids", _I32, (R,)),
            _want(row_lens, "row_lens", _I32, (R, P))), R, P, Hq


def _attn_out(q, out, out_lse, workspace):
    """The arguments the two attention calls end with, before the stream."""
    return (_want(out, "out", _BF16, q.shape),
            None if out_lse is None else _want(out_lse, "out_lse", _F32, q.shape[:3]),
            _dev(workspace, "workspace"), workspace.nbytes)


def idx_attn_paged(q, k_payload, k_scale, v_payload, v_scale, kv_dtype: str, page_table, slot_ids,
                   row_lens, kv_heads: int, sm_scale: float, out, out_lse, workspace,
                   stream=None) -> None:
    """Attention of q [R, P, q_heads, 128] over the whole paged cache into out (and
    out_lse, fp32 [R, P, q_heads], or None).  Planes: [num_pages * kv_heads * 64,
    128] rows with head page p * kv_heads + h; scales (fp8_e4m3 only) fp32 [rows]."""
    head, R, P, Hq = _attn_args(q, k_payload, k_scale, v_payload, v_scale, kv_dtype, page_table,
                                slot_ids, row_lens, kv_heads)
    tail = _attn_out(q, out, out_lse, workspace)
    _one_device(stream, q, k_payload, k_scale, v_payload, v_scale, page_table, slot_ids, row_lens, out,
                out_lse, workspace)
    rc = lib().idx_attn_paged(*head, R, P, Hq, sm_scale, *tail, _stream_of(q, stream))
    if rc:
        _check(rc, "idx_attn_paged")


def idx_attn_blocks(q, k_payload, k_scale, v_payload, v_scale, kv_dtype: str, page_table, slot_ids,
                    row_lens, block_ids, lists: int, kv_heads: int, sm_scale: float, out, out_lse,
                    workspace, stream=None) -> None:
    """idx_attn_paged over the 128-token blocks of block_ids [R, P * lists, topk]
    (idx_score_topk's out_ids with gqa = lists)."""
    if block_ids is None or block_ids.dim() != 3 or lists < 1:
        raise IdxError("block_ids must be [requests, draft rows * lists, topk] and lists >= 1")
    head, R, P, Hq = _attn_args(q, k_payload, k_scale, v_payload, v_scale, kv_dtype, page_table,
                                slot_ids, row_lens, kv_heads)
    topk = block_ids.shape[2]
    ids = _want(block_ids, "block_ids", _I32, (R, P * lists, topk))
    tail = _attn_out(q, out, out_lse, workspace)
    _one_device(stream, q, k_payload, k_scale, v_payload, v_scale, page_table, slot_ids, row_lens,
                block_ids, out, out_lse, workspace)
    rc = lib().idx_attn_blocks(*head, ids, lists, topk, R, P, Hq, sm_scale, *tail, _stream_of(q, stream))
    if rc:
        _check(rc, "idx_attn_blocks")


def idx_attn_paged_nvfp4(q, k_payload, k_scale, v_payload, v_scale, page_table, slot_ids, row_lens,
                         kv_heads: int, sm_scale: float, out, out_lse, workspace, k_outer: float = 1.0,
                         v_outer: float = 1.0, stream=None) -> None:
    """idx_attn_paged over NVFP4 planes (as for idx_store_kv_nvfp4)."""
    head, R, P, Hq = _attn_args(q, k_payload, k_scale, v_payload, v_scale, None, page_table, slot_ids,
                                row_lens, kv_heads)
    tail = _attn_out(q, out, out_lse, workspace)
    _one_device(stream, q, k_payload, k_scale, v_payload, v_scale, page_table, slot_ids, row_lens, out,
                out_lse, workspace)
    rc = lib().idx_attn_paged_nvfp4(*head, R, P, Hq, sm_scale, k_outer, v_outer, *tail, _stream_of(q, stream))
    if rc:
        _check(rc, "idx_attn_paged_nvfp4")


def idx_attn_blocks_nvfp4(q, k_payload, k_scale, v_payload, v_scale, page_table, slot_ids, row_lens,
                          block_ids, lists: int, kv_heads: int, sm_scale: float, out, out_lse, workspace,
                          k_outer: float = 1.0, v_outer: float = 1.0, stream=None) -> None:
    """idx_attn_blocks over NVFP4 planes (as for idx_store_kv_nvfp4)."""
    if block_ids is None or block_ids.dim() != 3 or lists < 1:
        raise IdxError("block_ids must be [requests, draft rows * lists, topk] and lists >= 1")
    head, R, P, Hq = _attn_args(q, k_payload, k_scale, v_payload, v_scale, None, page_table, slot_ids,
                                row_lens, kv_heads)
    topk = block_ids.shape[2]
    ids = _want(block_ids, "block_ids", _I32, (R, P * lists, topk))
    tail = _attn_out(q, out, out_lse, workspace)
    _one_device(stream, q, k_payload, k_scale, v_payload, v_scale, page_table, slot_ids, row_lens,
                block_ids, out, out_lse, workspace)
    rc = lib().idx_attn_blocks_nvfp4(*head, ids, lists, topk, R, P, Hq, sm_scale, k_outer, v_outer, *tail,
                                     _stream_of(q, stream))
    if rc:
        _check(rc, "idx_attn_blocks_nvfp4")


def idx_add_rmsnorm_fp8(x, residual, weight, eps: float, group: int, out, out_scale,
                        out_residual=None, stream=None) -> None:
    """x, residual (or None): bf16 [rows, dim], rows any stride apart; out: e4m3 codes
    [rows, dim]; out_scale: fp32, one per row (group 0) or per 128 elements;
    out_residual: bf16 [rows, dim], may be residual itself."""
    if x.dim() != 2:
        raise IdxError("x must be [rows, dim]")
    T, n = x.shape
    xp, xs = _rows_2d(x, "x", T, n)
    rp, rs = (None, 0) if residual is None else _rows_2d(residual, "residual", T, n)
    if out.dtype is not torch.float8_e4m3fn and out.dtype is not torch.uint8 or out.shape != (T, n):
        raise IdxError(f"out must be float8_e4m3fn or uint8 [{T}, {n}]")
    groups = -(-n // group) if group > 0 else 1
    if out_scale.dtype is not _F32 or out_scale.numel() != T * groups:
        raise IdxError(f"out_scale must be float32 [{T}, {groups}]")
    outs = (_dev(out, "out"), _dev(out_scale, "out_scale"),
            None if out_residual is None else _want(out_residual, "out_residual", _BF16, (T, n)))
    weight_ptr = _want(weight, "weight", _BF16, (n,))
    _one_device(stream, x, residual, weight, out, out_scale, out_residual)
    rc = lib().idx_add_rmsnorm_fp8(xp, xs, rp, rs, weight_ptr, T, n, group, eps, *outs,
                                   _stream_of(x, stream))
    if rc:
        _check(rc, "idx_add_rmsnorm_fp8")


NATIVE_CALLS = ("idx_attn_paged", "idx_attn_blocks", "idx_store_kv", "idx_add_rmsnorm_fp8",
                "idx_attn_paged_nvfp4", "idx_attn_blocks_nvfp4", "idx_store_kv_nvfp4", "idx_norm_rope_store")


def _native_calls():
    """The small-call operators of the CPython module, or these functions themselves
    where it has not been built (or torch lacks the bare stream call): the same checks and
    the same library calls, slower on the host."""
    here = tuple(globals()[name] for name in NATIVE_CALLS)
    if _raw_stream is None or not os.path.exists(LIB_PATH):
        return here
    try:
        from . import _binding
        _binding.bind((torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8,
                       torch.float8_e4m3fn), _raw_stream, _current_device, _check, here)
        return tuple(getattr(_binding, name) for name in NATIVE_CALLS)
    except (ImportError, TypeError, AttributeError):
        return here    # not built, built for another interpreter or from another state of the sources
