"""Python binding of libpagedattn, the sm_103a paged KV-cache attention library.

Argument marshalling only: each function reads shapes, dtypes and data pointers off torch
tensors and calls the C entry point of the same name declared in include/pa.h.  Every
step of the path runs in the library's CUDA kernels; there is no CPU or PyTorch
fallback, and a missing or unloadable library raises.

Tensors must be contiguous CUDA tensors on the current device.  Calls are asynchronous on
the current torch stream unless `stream` (a torch.cuda.Stream) is given.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Sequence

import torch

from .build import LIB as LIB_PATH

__all__ = [
    "PA_F32", "PA_F16", "PA_BF16", "PaError", "lib", "dtype_code",
    "slot_mapping", "reshape_and_cache", "cache_append", "copy_blocks", "swap_blocks",
    "decode_workspace_bytes",
    "decode", "decode_shared_prefix_workspace_bytes", "decode_shared_prefix",
    "prefill_workspace_bytes", "prefill_chunk", "get_status", "version",
    "set_stream_status", "release_thread_resources",
    "Rotary", "rotary_append", "decode_mass_workspace_bytes", "decode_mass",
    "prefill_mass_workspace_bytes", "prefill_mass", "evict_workspace_bytes", "evict",
    "testing_decode_workspace_bytes", "testing_decode_partitions",
    "STATUS_BAD_BLOCK", "STATUS_BAD_SLOT", "STATUS_BAD_CONTEXT", "STATUS_TIMEOUT", "STATUS_RANGE",
]

PA_F32, PA_F16, PA_BF16 = 0, 1, 2
STATUS_BAD_BLOCK, STATUS_BAD_SLOT, STATUS_BAD_CONTEXT, STATUS_TIMEOUT = 0x1, 0x2, 0x4, 0x8
STATUS_RANGE = 0x10  # reserved: no longer set
_ERRORS = {1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_WORKSPACE",
           4: "PA_ERR_CUDA"}

_DT = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}


class PaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_ERRORS.get(code, code)}: {msg}")
        self.code = code


_lib = None
_lock = threading.Lock()

_i, _u64, _f, _p, _sz = ctypes.c_int, ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_i64 = ctypes.c_int64

_SIGNATURES = {
    "pa_version": ([], _i),
    "pa_last_error_string": ([], ctypes.c_char_p),
    "pa_get_status": ([_p], _i),
    "pa_set_stream_status": ([_p, _p], _i),
    "pa_release_thread_resources": ([], _i),
    "pa_testing_decode_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i], _sz),
    "pa_testing_decode_partitions": ([_p, _i, _p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i,
                                      _i, _f, _i, _i, _p, _sz, _p], _i),
    "pa_selftest_wait_timeout": ([_i, _p], _i),
    "pa_mixed_step": ([_p, _p, _p, _p, _i, _i, _i, _i, _i, _f, _i, _p], _i),
    "pa_slot_mapping": ([_p, _p, _i, _p, _p, _i, _i, _i, _i, _p], _i),
    "pa_reshape_and_cache": ([_p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _p], _i),
    "pa_copy_blocks": ([_p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _p], _i),
    "pa_swap_blocks": ([_p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _i, _p], _i),
    "pa_cache_append": ([_p, _p, _p, _p, _p, _p, _i, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i,
                         _p], _i),
    "pa_decode_workspace_bytes": ([_i, _i, _i, _i, _i, _i], _sz),
    "pa_decode_shared_prefix_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i, _i], _sz),
    "pa_decode_shared_prefix": ([_p, _i, _p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _i,
                                 _p, _i, _p, _i, _f, _i, _p, _sz, _p], _i),
    "pa_decode": ([_p, _i, _p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz,
                   _p], _i),
    "pa_decode_append": ([_p, _i, _p, _p, _p, _p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i,
                          _i, _f, _i, _p, _sz, _p], _i),
    "pa_prefill_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i, _i], _sz),
    "pa_prefill_chunk": ([_p, _i, _p, _p, _p, _p, _i, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i,
                          _i, _f, _i, _p, _sz, _p], _i),
    "pa_rotary_append": ([_p, _p, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p, _i, _p, _p, _p, _i,
                          _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _p], _i),
    "pa_decode_mass_workspace_bytes": ([_i, _i, _i, _i, _i, _i], _sz),
    "pa_decode_mass": ([_p, _i, _p, _p, _p, _p, _i, _p, _i, _p, _i64, _p, _i, _f, _i, _i, _i, _i,
                        _i, _i, _f, _i, _p, _sz, _p], _i),
    "pa_prefill_mass_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i, _i], _sz),
    "pa_prefill_mass": ([_p, _i, _p, _p, _p, _p, _i, _p, _p, _p, _i, _i, _p, _i64, _p, _i, _f,
                         _i, _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p], _i),
    "pa_evict_workspace_bytes": ([_i, _i, _i, _i], _sz),
    "pa_evict": ([_p, _p, _p, _p, _i64, _p, _i, _p, _i, _p, _i, _p, _p, _i, _i, _i, _i, _p, _p,
                  _i, _i, _i, _i, _i, _i, _p, _sz, _p], _i),
}


def lib(path: Optional[str] = None):
    """Loads libpagedattn.so once (raising if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise ImportError(
                    f"libpagedattn.so is not built ({p}); build it with "
                    "`python -m paged_kv_cache_53_gb300.build`")
            handle = ctypes.CDLL(p)
            for name, (args, res) in _SIGNATURES.items():
                fn = getattr(handle, name)
                fn.argtypes = args
                fn.restype = res
            _lib = handle
    return _lib


def version() -> int:
    return lib().pa_version()


def _check(rc: int):
    if rc != 0:
        raise PaError(rc, lib().pa_last_error_string().decode())


def dtype_code(t: torch.dtype) -> int:
    try:
        return _DT[t]
    except KeyError:
        raise TypeError(f"unsupported dtype {t}") from None


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libpagedattn must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    # the handle of torch.cuda.current_stream() without the Stream object around it, which
    # takes a quarter of a small call's time
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _i32(t: torch.Tensor, name: str):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")


def slot_mapping(slots: torch.Tensor, block_tables: torch.Tensor, cu_q_lens: torch.Tensor,
                 context_lens: torch.Tensor, block_size: int, num_blocks: int, stream=None):
    """slots[t] (int64) = physical slot of new token t (see pa_slot_mapping)."""
    _i32(block_tables, "block_tables")
    if slots.dtype != torch.int64:
        raise TypeError("slots must be int64")
    _check(lib().pa_slot_mapping(_ptr(slots), _ptr(block_tables), block_tables.shape[1],
                                 _ptr(cu_q_lens), _ptr(context_lens), context_lens.shape[0],
                                 slots.shape[0], block_size, num_blocks, _stream(stream)))


def reshape_and_cache(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, slots: torch.Tensor, stream=None):
    """Writes k_new/v_new [T, H_kv, D] into the caches [NB, H_kv, BS, D] at `slots`."""
    nb, h_kv, bs, d = k_cache.shape
    _check(lib().pa_reshape_and_cache(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(slots), k_new.shape[0], h_kv, d, bs, nb,
                                      dtype_code(k_cache.dtype), _stream(stream)))


def cache_append(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, block_tables: torch.Tensor, cu_q_lens: torch.Tensor,
                 context_lens: torch.Tensor, max_q: int, slots: Optional[torch.Tensor] = None,
                 stream=None):
    """Slot mapping and cache write of the step's new tokens in one launch."""
    nb, h_kv, bs, d = k_cache.shape
    _i32(block_tables, "block_tables")
    if slots is not None and slots.dtype != torch.int64:
        raise TypeError("slots must be int64")
    _check(lib().pa_cache_append(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(slots), _ptr(block_tables), block_tables.shape[1],
                                 _ptr(cu_q_lens), _ptr(context_lens), context_lens.shape[0],
                                 k_new.shape[0], max_q, h_kv, d, bs, nb,
                                 dtype_code(k_cache.dtype), _stream(stream)))


def copy_blocks(k_caches: Sequence[torch.Tensor], v_caches: Sequence[torch.Tensor],
                pairs: torch.Tensor, stream=None):
    """Block dst <- block src for every (src, dst) row of `pairs`, in every layer."""
    n = len(k_caches)
    if n != len(v_caches) or n == 0:
        raise ValueError("need the same non-zero number of K and V caches")
    nb, h_kv, bs, d = k_caches[0].shape
    karr = (ctypes.c_void_p * n)(*[_ptr(t) for t in k_caches])
    varr = (ctypes.c_void_p * n)(*[_ptr(t) for t in v_caches])
    _check(lib().pa_copy_blocks(karr, varr, n, _ptr(pairs), pairs.shape[0], h_kv, d, bs, nb,
                                dtype_code(k_caches[0].dtype), _stream(stream)))


def swap_blocks(src_k: Sequence[torch.Tensor], src_v: Sequence[torch.Tensor],
                dst_k: Sequence[torch.Tensor], dst_v: Sequence[torch.Tensor],
                pairs: torch.Tensor, stream=None):
    """Block dst of every destination pool <- block src of the matching source pool, for
    every (src, dst) row of `pairs` (see pa_swap_blocks).  Pools are CUDA tensors or
    pinned CPU tensors of one geometry [blocks, H_kv, block_size, D]."""
    n = len(src_k)
    if not (n == len(src_v) == len(dst_k) == len(dst_v)) or n == 0:
        raise ValueError("need the same non-zero number of pools on every side")
    _i32(pairs, "pairs")
    if pairs.device.type == "cpu" and not pairs.is_pinned():
        raise ValueError("pairs must be a CUDA tensor or a pinned CPU tensor")
    nbs, h_kv, bs, d = src_k[0].shape
    nbd = dst_k[0].shape[0]
    arr = lambda ts: (ctypes.c_void_p * n)(*[_ptr(t) for t in ts])
    _check(lib().pa_swap_blocks(arr(src_k), arr(src_v), arr(dst_k), arr(dst_v), n, _ptr(pairs),
                                pairs.shape[0], h_kv, d, bs, nbs, nbd,
                                dtype_code(src_k[0].dtype), _stream(stream)))


def decode_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                           max_ctx: int, block_size: int) -> int:
    return int(lib().pa_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                               max_ctx, block_size))


def decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, context_lens: torch.Tensor, max_ctx: int, scale: float,
           workspace: torch.Tensor, stream=None):
    """Paged decode attention (see pa_decode); `workspace` is a uint8 device tensor of at
    least decode_workspace_bytes(...) bytes."""
    nb, h_kv, bs, d = k_cache.shape
    b, h_q, _ = q.shape
    _check(lib().pa_decode(_ptr(out), dtype_code(out.dtype), _ptr(q), _ptr(k_cache),
                           _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
                           _ptr(context_lens), max_ctx, b, h_q, h_kv, d, bs, nb, float(scale),
                           dtype_code(k_cache.dtype), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream)))


def decode_append(out: torch.Tensor, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, max_ctx: int, scale: float,
                  workspace: torch.Tensor, slots: Optional[torch.Tensor] = None, stream=None):
    """One decode step (see pa_decode_append): row b of k_new / v_new is written at
    position context_lens[b] - 1 of sequence b (its slot into `slots` if given), then the
    decode attends over every context."""
    nb, h_kv, bs, d = k_cache.shape
    b, h_q, _ = q.shape
    if slots is not None and slots.dtype != torch.int64:
        raise TypeError("slots must be int64")
    _check(lib().pa_decode_append(_ptr(out), dtype_code(out.dtype), _ptr(q), _ptr(k_new),
                                  _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(slots),
                                  _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                                  max_ctx, b, h_q, h_kv, d, bs, nb, float(scale),
                                  dtype_code(k_cache.dtype), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))


class _DecodeBatch(ctypes.Structure):
    """pa_decode_batch of include/pa.h."""
    _fields_ = [("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("q", ctypes.c_void_p),
                ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("block_tables", ctypes.c_void_p),
                ("max_blocks_per_seq", ctypes.c_int), ("context_lens", ctypes.c_void_p),
                ("max_ctx", ctypes.c_int), ("num_seqs", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class _PrefillBatch(ctypes.Structure):
    """pa_prefill_batch of include/pa.h."""
    _fields_ = [("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("q", ctypes.c_void_p),
                ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("block_tables", ctypes.c_void_p),
                ("max_blocks_per_seq", ctypes.c_int), ("cu_q_lens", ctypes.c_void_p),
                ("context_lens", ctypes.c_void_p), ("max_q", ctypes.c_int),
                ("max_ctx", ctypes.c_int), ("num_seqs", ctypes.c_int),
                ("num_tokens", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


def mixed_step(k_cache: torch.Tensor, v_cache: torch.Tensor, scale: float,
               decode: Optional[dict] = None, prefill: Optional[dict] = None, stream=None):
    """One step of a batch of decodes and prefill chunks run side by side (see
    pa_mixed_step).  `decode`: out, q, k_new, v_new, block_tables, context_lens, max_ctx,
    workspace[, slots]; `prefill`: the same plus cu_q_lens and max_q (k_new / v_new hold the
    chunks' new tokens)."""
    nb, h_kv, bs, d = k_cache.shape
    h_q = None
    dp = pp = None
    if decode is not None:
        m = decode
        h_q = m["q"].shape[1]
        ws = m["workspace"]
        dp = _DecodeBatch(_ptr(m["out"]), dtype_code(m["out"].dtype), _ptr(m["q"]),
                          _ptr(m["k_new"]), _ptr(m["v_new"]), _ptr(m.get("slots")),
                          _ptr(m["block_tables"]), m["block_tables"].shape[1],
                          _ptr(m["context_lens"]), int(m["max_ctx"]), m["q"].shape[0],
                          _ptr(ws), ws.numel() * ws.element_size())
    if prefill is not None:
        m = prefill
        h_q = m["q"].shape[1]
        ws = m["workspace"]
        pp = _PrefillBatch(_ptr(m["out"]), dtype_code(m["out"].dtype), _ptr(m["q"]),
                           _ptr(m["k_new"]), _ptr(m["v_new"]), _ptr(m.get("slots")),
                           _ptr(m["block_tables"]), m["block_tables"].shape[1],
                           _ptr(m["cu_q_lens"]), _ptr(m["context_lens"]), int(m["max_q"]),
                           int(m["max_ctx"]), m["cu_q_lens"].shape[0] - 1, m["q"].shape[0],
                           _ptr(ws), ws.numel() * ws.element_size())
    if h_q is None:
        return
    _check(lib().pa_mixed_step(ctypes.byref(dp) if dp is not None else None,
                               ctypes.byref(pp) if pp is not None else None, _ptr(k_cache),
                               _ptr(v_cache), h_q, h_kv, d, bs, nb, float(scale),
                               dtype_code(k_cache.dtype), _stream(stream)))


def decode_shared_prefix_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                         head_dim: int, max_ctx: int, block_size: int,
                                         num_sharers: int, prefix_len: int) -> int:
    return int(lib().pa_decode_shared_prefix_workspace_bytes(
        num_seqs, num_q_heads, num_kv_heads, head_dim, max_ctx, block_size, num_sharers,
        prefix_len))


def decode_shared_prefix(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, block_tables: torch.Tensor,
                         context_lens: torch.Tensor, max_ctx: int, prefix_blocks: torch.Tensor,
                         prefix_len: int, sharers: torch.Tensor, scale: float,
                         workspace: torch.Tensor, stream=None):
    """pa_decode with the prefix shared by the rows in `sharers` attended once per KV head
    (see pa_decode_shared_prefix)."""
    nb, h_kv, bs, d = k_cache.shape
    b, h_q, _ = q.shape
    _i32(prefix_blocks, "prefix_blocks")
    _i32(sharers, "sharers")
    _check(lib().pa_decode_shared_prefix(
        _ptr(out), dtype_code(out.dtype), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), max_ctx, b, h_q, h_kv, d,
        bs, nb, _ptr(prefix_blocks), prefix_len, _ptr(sharers), sharers.shape[0], float(scale),
        dtype_code(k_cache.dtype), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def prefill_workspace_bytes(num_seqs: int, num_tokens: int, max_q: int, num_q_heads: int,
                            num_kv_heads: int, head_dim: int, max_ctx: int,
                            block_size: int) -> int:
    return int(lib().pa_prefill_workspace_bytes(num_seqs, num_tokens, max_q, num_q_heads,
                                                num_kv_heads, head_dim, max_ctx, block_size))


def prefill_chunk(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, block_tables: torch.Tensor, cu_q_lens: torch.Tensor,
                  context_lens: torch.Tensor, max_q: int, max_ctx: int, scale: float,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Causal chunked-prefill attention over paged context (see pa_prefill_chunk)."""
    nb, h_kv, bs, d = k_cache.shape
    t, h_q, _ = q.shape
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().pa_prefill_chunk(_ptr(out), dtype_code(out.dtype), _ptr(q), _ptr(k_cache),
                                  _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
                                  _ptr(cu_q_lens), _ptr(context_lens), context_lens.shape[0], t,
                                  max_q, max_ctx, h_q, h_kv, d, bs, nb, float(scale),
                                  dtype_code(k_cache.dtype), ws_ptr, ws_bytes, _stream(stream)))


class Rotary:
    """Frequencies and axes of rotary positions (see pa_rotary_append), laid out once.

    inv_freq: radians per position of each pair; its length is rotary_dim / 2.  pair_axis: the
    position axis of each pair (0 for all when omitted).  interleaved: pairs are neighbouring
    elements instead of the two halves of the first rotary_dim elements."""

    def __init__(self, inv_freq: Sequence[float], pair_axis: Optional[Sequence[int]] = None,
                 interleaved: bool = False):
        n = len(inv_freq)
        if n == 0:
            raise ValueError("inv_freq is empty")
        if pair_axis is not None and len(pair_axis) != n:
            raise ValueError(f"{len(pair_axis)} axes for {n} pairs")
        self.rotary_dim = 2 * n
        self.interleaved = int(bool(interleaved))
        self.inv_freq = (ctypes.c_double * n)(*[float(f) for f in inv_freq])
        self.pair_axis = (ctypes.c_int32 * n)(*([int(a) for a in pair_axis] if pair_axis is not None
                                                else [0] * n))


def _token_rows(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str):
    """Pointer and token stride of a [tokens, heads, dim] tensor whose rows are contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    stride, heads, elem = t.stride()
    if shape[0] > 0 and (elem != 1 or (heads != shape[2] and shape[1] > 1)):
        raise ValueError(f"{name} must have contiguous rows of heads")
    return t.data_ptr(), stride if shape[0] > 1 else shape[1] * shape[2]


def rotary_append(q_out: torch.Tensor, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  cu_q_lens: Optional[torch.Tensor], context_lens: torch.Tensor,
                  positions: torch.Tensor, rotary: Rotary, slots: Optional[torch.Tensor] = None,
                  stream=None):
    """Rotary positions of a step's queries and keys, and the cache write of the turned keys and
    the values (see pa_rotary_append).  q, k_new, v_new [T, H, D] may be views with a token
    stride; positions int32 [axes, T]; cu_q_lens None: one new token per sequence."""
    cache, rows = k_cache.shape, q.shape
    nb, h_kv, bs, d = cache
    dtype = k_cache.dtype
    if len(rows) != 3:
        raise ValueError("q must be [tokens, heads, dim]")
    t, h_q, _ = rows
    qp, qs = _token_rows(q, dtype, (t, h_q, d), "q")
    kp, ks = _token_rows(k_new, dtype, (t, h_kv, d), "k_new")
    vp, vs = _token_rows(v_new, dtype, (t, h_kv, d), "v_new")
    if q_out.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError(f"q_out and the caches must be {dtype}")
    if q_out.shape != rows or v_cache.shape != cache:
        raise ValueError("q_out must be like q, and the caches alike")
    i32 = torch.int32
    if (block_tables.dtype != i32 or context_lens.dtype != i32 or positions.dtype != i32 or
            (cu_q_lens is not None and cu_q_lens.dtype != i32)):
        raise TypeError("block_tables, cu_q_lens, context_lens and positions must be int32")
    b = context_lens.shape[0]
    axes = positions.shape
    if len(axes) != 2 or axes[1] != t:
        raise ValueError("positions must be [axes, tokens]")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != b:
        raise ValueError("block_tables must have a row per sequence")
    if cu_q_lens is not None:
        if cu_q_lens.shape[0] != b + 1:
            raise ValueError("cu_q_lens must have one entry more than context_lens")
    elif t > b:
        raise ValueError("without cu_q_lens there is one token per sequence")
    if slots is not None and (slots.dtype != torch.int64 or slots.numel() < t):
        raise TypeError("slots must be int64 [tokens]")
    _check(lib().pa_rotary_append(
        _ptr(q_out), qp, qs, kp, ks, vp, vs, _ptr(k_cache), _ptr(v_cache), _ptr(slots),
        _ptr(block_tables), tables[1], _ptr(cu_q_lens), _ptr(context_lens),
        _ptr(positions), axes[0], rotary.inv_freq, rotary.pair_axis,
        rotary.rotary_dim, rotary.interleaved, b, t, h_q, h_kv, d, bs, nb, dtype_code(dtype),
        _stream_for(stream, q_out, q, k_new, v_new, k_cache, v_cache, block_tables, cu_q_lens,
                    context_lens, positions, slots)))


def _stream_for(stream, *tensors: Optional[torch.Tensor]) -> int:
    """The stream's handle; every tensor of the call has to be on the current device, since
    the kernels take its address as it is."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"the tensors must be on the current device (cuda:{device}): one of "
                             f"{t.dtype} {list(t.shape)} is on {t.device}")
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)


def _attention_args(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, block_tables: torch.Tensor,
                    context_lens: torch.Tensor):
    """Shapes and types that the C call cannot see.  Returns the shapes of q, the caches and the
    block tables, and the number of sequences."""
    rows, cache, tables, b = q.shape, k_cache.shape, block_tables.shape, context_lens.shape[0]
    if len(rows) != 3 or out.shape != rows or rows[2] != cache[3]:
        raise ValueError("q and out must be [tokens, heads, dim] alike, dim that of the caches")
    if v_cache.shape != cache:
        raise ValueError("the two caches must be alike")
    if not q.dtype == v_cache.dtype == k_cache.dtype:
        raise TypeError("q and the caches must have one type")
    if not block_tables.dtype == context_lens.dtype == torch.int32:
        raise TypeError("block_tables and context_lens must be int32")
    if len(tables) != 2 or tables[0] != b:
        raise ValueError("block_tables must have a row per sequence")
    return rows, cache, tables, b


def _mass(mass: torch.Tensor, mass_rows: Optional[torch.Tensor], h_kv: int, b: int):
    """(pointer, stride, rows pointer, rows) of a [rows, H_kv, positions] mass."""
    shape = mass.shape
    if mass.dtype != torch.float32 or len(shape) != 3 or shape[1] != h_kv:
        raise TypeError("mass must be float32 [rows, H_kv, positions]")
    if mass_rows is not None:
        _i32(mass_rows, "mass_rows")
        if mass_rows.numel() != b:
            raise ValueError("mass_rows must have one entry per sequence")
    return _ptr(mass), shape[2], _ptr(mass_rows), shape[0]


def decode_mass_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                max_ctx: int, block_size: int) -> int:
    return int(lib().pa_decode_mass_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                    max_ctx, block_size))


def decode_mass(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                block_tables: torch.Tensor, context_lens: torch.Tensor, max_ctx: int,
                scale: float, mass: torch.Tensor, workspace: torch.Tensor,
                mass_rows: Optional[torch.Tensor] = None, decay: float = 1.0, stream=None):
    """Paged decode attention that also adds every position's attention weight to `mass`
    (float32 [rows, H_kv, positions], see pa_decode_mass)."""
    (t, h_q, _), (nb, h_kv, bs, d), tables, b = _attention_args(out, q, k_cache, v_cache,
                                                                 block_tables, context_lens)
    if t != b:
        raise ValueError("q must have a row per sequence")
    m, ms, mr, nr = _mass(mass, mass_rows, h_kv, b)
    _check(lib().pa_decode_mass(_ptr(out), dtype_code(out.dtype), _ptr(q), _ptr(k_cache),
                                _ptr(v_cache), _ptr(block_tables), tables[1],
                                _ptr(context_lens), max_ctx, m, ms, mr, nr, float(decay), b, h_q,
                                h_kv, d, bs, nb, float(scale), dtype_code(k_cache.dtype),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream_for(stream, out, q, k_cache, v_cache, block_tables,
                                            context_lens, mass, mass_rows, workspace)))


def prefill_mass_workspace_bytes(num_seqs: int, num_tokens: int, max_q: int, num_q_heads: int,
                                 num_kv_heads: int, head_dim: int, max_ctx: int,
                                 block_size: int) -> int:
    return int(lib().pa_prefill_mass_workspace_bytes(num_seqs, num_tokens, max_q, num_q_heads,
                                                     num_kv_heads, head_dim, max_ctx, block_size))


def prefill_mass(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_tables: torch.Tensor, cu_q_lens: torch.Tensor, context_lens: torch.Tensor,
                 max_q: int, max_ctx: int, scale: float, mass: torch.Tensor,
                 workspace: torch.Tensor, observe: Optional[torch.Tensor] = None,
                 mass_rows: Optional[torch.Tensor] = None, decay: float = 1.0, stream=None):
    """Causal chunked-prefill attention that also adds the weights its queries (or, with
    `observe`, the last observe[b] of each chunk) give every position to `mass` (see
    pa_prefill_mass)."""
    (t, h_q, _), (nb, h_kv, bs, d), tables, b = _attention_args(out, q, k_cache, v_cache,
                                                                 block_tables, context_lens)
    _i32(cu_q_lens, "cu_q_lens")
    if cu_q_lens.shape[0] != b + 1:
        raise ValueError("cu_q_lens must have one entry more than context_lens")
    m, ms, mr, nr = _mass(mass, mass_rows, h_kv, b)
    if observe is not None:
        _i32(observe, "observe")
        if observe.numel() != b:
            raise ValueError("observe must have one entry per sequence")
    _check(lib().pa_prefill_mass(_ptr(out), dtype_code(out.dtype), _ptr(q), _ptr(k_cache),
                                 _ptr(v_cache), _ptr(block_tables), tables[1],
                                 _ptr(cu_q_lens), _ptr(context_lens), _ptr(observe), max_q,
                                 max_ctx, m, ms, mr, nr, float(decay), b, t, h_q, h_kv, d, bs, nb,
                                 float(scale), dtype_code(k_cache.dtype), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(),
                                 _stream_for(stream, out, q, k_cache, v_cache, block_tables,
                                             cu_q_lens, context_lens, observe, mass, mass_rows,
                                             workspace)))


def evict_workspace_bytes(num_seqs: int, num_kv_heads: int, max_ctx: int, max_keep: int) -> int:
    return int(lib().pa_evict_workspace_bytes(num_seqs, num_kv_heads, max_ctx, max_keep))


def evict(k_cache: torch.Tensor, v_cache: torch.Tensor, mass: torch.Tensor,
          new_mass: torch.Tensor, block_tables: torch.Tensor, new_block_tables: torch.Tensor,
          context_lens: torch.Tensor, keep_lens: torch.Tensor, max_ctx: int,
          new_context_lens: torch.Tensor, kept: torch.Tensor, workspace: torch.Tensor,
          sinks: int = 0, recent: int = 0, mass_rows: Optional[torch.Tensor] = None, stream=None):
    """Cuts every sequence's cache down to its keep_lens[b] weightiest positions per KV head,
    in place or into new blocks (see pa_evict).  `kept` int32 [sequences, H_kv, max_keep]
    receives the kept positions, new_context_lens the new lengths."""
    cache, tables, new_tables = k_cache.shape, block_tables.shape, new_block_tables.shape
    nb, h_kv, bs, d = cache
    b, lists = context_lens.shape[0], kept.shape
    i32 = torch.int32
    if not (block_tables.dtype == new_block_tables.dtype == context_lens.dtype ==
            keep_lens.dtype == new_context_lens.dtype == kept.dtype == i32):
        raise TypeError("tables, lengths and kept must be int32")
    if (len(tables) != 2 or len(new_tables) != 2 or
            not tables[0] == new_tables[0] == keep_lens.shape[0] == new_context_lens.shape[0] == b):
        raise ValueError("tables and lengths must have an entry per sequence")
    if len(lists) != 3 or lists[0] != b or lists[1] != h_kv:
        raise ValueError("kept must be [sequences, H_kv, max_keep]")
    if new_mass.shape != mass.shape or new_mass.dtype != mass.dtype:
        raise ValueError("new_mass must be like mass")
    if v_cache.shape != cache or v_cache.dtype != k_cache.dtype:
        raise ValueError("the two caches must be alike")
    m, ms, mr, nr = _mass(mass, mass_rows, h_kv, b)
    _check(lib().pa_evict(_ptr(k_cache), _ptr(v_cache), m, _ptr(new_mass), ms, mr, nr,
                          _ptr(block_tables), tables[1], _ptr(new_block_tables),
                          new_tables[1], _ptr(context_lens), _ptr(keep_lens), max_ctx,
                          lists[2], int(sinks), int(recent), _ptr(new_context_lens),
                          _ptr(kept), b, h_kv, d, bs, nb, dtype_code(k_cache.dtype),
                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                          _stream_for(stream, k_cache, v_cache, mass, new_mass, block_tables,
                                      new_block_tables, context_lens, keep_lens,
                                      new_context_lens, kept, mass_rows, workspace)))


def testing_decode_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                   head_dim: int, max_ctx: int, block_size: int,
                                   part_blocks: int) -> int:
    return int(lib().pa_testing_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads,
                                                       head_dim, max_ctx, block_size,
                                                       part_blocks))


def testing_decode_partitions(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                              v_cache: torch.Tensor, block_tables: torch.Tensor,
                              context_lens: torch.Tensor, max_ctx: int, scale: float,
                              part_blocks: int, workspace: torch.Tensor, stream=None):
    """pa_decode with every context cut into partitions of `part_blocks` blocks (see
    pa_testing_decode_partitions in include/pa_testing.h)."""
    nb, h_kv, bs, d = k_cache.shape
    b, h_q, _ = q.shape
    _check(lib().pa_testing_decode_partitions(
        _ptr(out), dtype_code(out.dtype), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), max_ctx, b, h_q, h_kv, d,
        bs, nb, float(scale), dtype_code(k_cache.dtype), int(part_blocks), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def set_stream_status(stream, status: Optional[torch.Tensor]):
    """Routes the status bits of calls on `stream` (a torch.cuda.Stream) into `status`, a
    one-element int32 CUDA tensor the caller reads and clears; None removes the route
    (see pa_set_stream_status)."""
    if status is not None:
        if status.dtype != torch.int32 or status.device.type != "cuda" or status.numel() < 1:
            raise TypeError("status must be an int32 CUDA tensor")
    _check(lib().pa_set_stream_status(_stream(stream), _ptr(status)))


def release_thread_resources():
    """Destroys the side stream and events pa_mixed_step created for this thread."""
    _check(lib().pa_release_thread_resources())


def get_status() -> int:
    """Reads and clears the device status word (synchronises the device)."""
    v = ctypes.c_int32(0)
    _check(lib().pa_get_status(ctypes.byref(v)))
    return int(v.value)


def selftest_wait_timeout(timeout_us: int, stream=None):
    """Runs the bounded-wait self-test: one kernel waits on an mbarrier nothing arrives
    on, gives up after `timeout_us` microseconds and sets STATUS_TIMEOUT."""
    _check(lib().pa_selftest_wait_timeout(int(timeout_us), _stream(stream)))
