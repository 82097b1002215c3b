"""ctypes binding of libpa.so: argument marshalling only.

Every function checks the torch tensors it is given (device, dtype,
contiguity), passes raw device pointers and the current CUDA stream to the C
ABI declared in ``include/pa.h``, and raises ``PagedAttentionError`` on a
non-zero status.  All arithmetic happens in the library's CUDA kernels; there
is no CPU fallback -- importing this module raises ImportError when libpa.so
has not been built.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpa.so")

PA_F32, PA_BF16 = 0, 1
PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA, PA_ERR_DEVICE_INDEX = 0, 1, 2, 3, 4, 5
DEVERR_BLOCK_ID, DEVERR_SLOT, DEVERR_CONTEXT, DEVERR_COPY, DEVERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8, 0x10
PHASE_PLAN, PHASE_ATTEND, PHASE_REDUCE, PHASE_ALL = 0x1, 0x2, 0x4, 0x7

_vp, _i, _i32p, _i64p, _sz, _f = (ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_size_t, ctypes.c_float)

_DECODE_ARGS = [_vp, _i, _vp, _vp, _vp, _i32p, _i32p, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i,
                _vp, _sz, _i, _i32p, _vp]

SIGNATURES = {
    "pa_reshape_and_cache": (_i, [_vp, _vp, _vp, _vp, _i64p, _i, _i, _i, _i, _i, _i, _i32p, _vp]),
    "pa_decode_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "pa_decode": (_i, _DECODE_ARGS),
    "pa_decode_phases": (_i, _DECODE_ARGS + [_i]),
    "pa_decode_step": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _i64p, _i, _i64p, _i, _i32p, _i32p, _i, _i, _i, _i,
                            _i, _i, _i, _i, _f, _i, _vp, _sz, _i, _i32p, _vp]),
    "pa_copy_blocks": (_i, [_vp, _vp, _i64p, _i, _sz, _i, _i32p, _vp]),
    "pa_prefill_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "pa_prefill_uses_tensor_cores": (_i, [_i, _i, _i, _i, _i]),
    "pa_prefill": (_i, [_vp, _i, _vp, _vp, _vp, _i32p, _i32p, _i32p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                        _i, _vp, _sz, _i, _i32p, _vp]),
    "pa_decode_noalloc": (_i, [_vp, _i, _vp, _vp, _vp, _i32p, _i32p, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                               _i, _i, _i32p, _vp]),
    "pa_tree_workspace_bytes": (_sz, [_i, _i, _i]),
    "pa_tree_uses_tensor_cores": (_i, [_i, _i]),
    "pa_tree_decode": (_i, [_vp, _i, _vp, _vp, _vp, _i32p, _i32p, _i32p, _i64p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                            _f, _vp, _sz, _i, _i32p, _vp]),
    "pa_tree_mask": (_i, [_vp, _i, _i, _vp]),
    "pa_decode_weights_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "pa_decode_weights": (_i, [_vp, _i, _vp, _vp, _i32p, _i, _vp, _vp, _vp, _i32p, _i32p, _i, _i, _i, _i, _i, _i, _i,
                               _i, _f, _i, _vp, _sz, _i, _i32p, _vp]),
    "pa_select_tokens": (_i, [_i32p, _i32p, _vp, _i32p, _i32p, _i, _i, _i, _i, _i, _i32p, _vp]),
    "pa_compact": (_i, [_vp, _vp, _vp, _vp, _i, _i32p, _i32p, _i, _i, _i32p, _i, _i, _i32p, _i32p, _i, _i, _i, _i, _i,
                        _i, _i32p, _vp]),
    "pa_bm_create": (ctypes.c_void_p, [_i, _i, _vp, _i]),
    "pa_bm_destroy": (None, [_vp]),
    "pa_bm_add_sequence": (_i, [_vp, ctypes.c_int64]),
    "pa_bm_fork": (_i, [_vp, ctypes.c_int64, ctypes.c_int64]),
    "pa_bm_free": (_i, [_vp, ctypes.c_int64]),
    "pa_bm_append": (_i, [_vp, ctypes.c_int64, _vp, _i, _vp, _vp, _i, ctypes.POINTER(ctypes.c_int),
                          ctypes.POINTER(ctypes.c_int)]),
    "pa_bm_append_batch": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _i, ctypes.POINTER(ctypes.c_int),
                                ctypes.POINTER(ctypes.c_int)]),
    "pa_bm_compact": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(ctypes.c_int)]),
    "pa_bm_block_table": (_i, [_vp, ctypes.c_int64, _vp, _i, ctypes.POINTER(ctypes.c_int),
                               ctypes.POINTER(ctypes.c_int64)]),
    "pa_bm_num_free": (_i, [_vp]),
    "pa_bm_ref_count": (_i, [_vp, _i]),
    "pa_selftest_bounded_wait": (_i, [_i32p, ctypes.c_uint64, _vp]),
    "pa_status_string": (ctypes.c_char_p, [_i]),
    "pa_version": (_i, []),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built: run `python -m paged_kv_cache_382_b200.build` "
            "(needs nvcc); this package has no CPU fallback")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (restype, argtypes) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = restype
        fn.argtypes = argtypes
    return lib


lib = _load()


class PagedAttentionError(RuntimeError):
    def __init__(self, what: str, status: int):
        super().__init__(f"{what}: {lib.pa_status_string(status).decode()}")
        self.status = status


def _check(status: int, what: str) -> None:
    if status != PA_OK:
        raise PagedAttentionError(what, status)


def dtype_code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return PA_F32
    if dtype == torch.bfloat16:
        return PA_BF16
    raise TypeError(f"unsupported dtype {dtype}; the kernels take float32 or bfloat16")


# The current stream's handle without building a Stream object (3 us of a call's 12).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _allocating_for(stream: Optional[torch.cuda.Stream]):
    """Context in which a call launched on ``stream`` allocates what it drops on return: memory of that
    stream, which nobody else gets before the call's kernels are through with it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _opt_err(dev_err: Optional[torch.Tensor]) -> Optional[int]:
    if dev_err is None:
        return None
    return _dev(dev_err, "dev_err", torch.int32)


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                      dev_err: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write key/value [T][Hkv][d] into the pools [NB][Hkv][B][d] at slot_mapping (int64 [T])."""
    NB, Hkv, B, d = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache must have the same shape")
    T = key.shape[0]
    if tuple(key.shape) != (T, Hkv, d) or tuple(value.shape) != (T, Hkv, d):
        raise ValueError("key/value must be [num_tokens][num_kv_heads][head_dim]")
    if tuple(slot_mapping.shape) != (T,):
        raise ValueError("slot_mapping must be [num_tokens]")
    dt = k_cache.dtype
    rc = lib.pa_reshape_and_cache(
        _dev(key, "key", dt), _dev(value, "value", dt), _dev(k_cache, "k_cache", dt),
        _dev(v_cache, "v_cache", dt), _dev(slot_mapping, "slot_mapping", torch.int64), T, Hkv, d, B,
        NB, dtype_code(dt), _opt_err(dev_err), _stream_handle(stream))
    _check(rc, "pa_reshape_and_cache")


def decode_workspace_bytes(num_seqs: int, num_heads: int, head_dim: int, max_context_len: int,
                           partition_size: int = 512) -> int:
    n = lib.pa_decode_workspace_bytes(num_seqs, num_heads, head_dim, max_context_len, partition_size)
    if n == 0:
        raise ValueError("invalid arguments for pa_decode_workspace_bytes")
    return int(n)


def decode_capacity(block_tables: torch.Tensor, block_size: int, max_context_len: int = 0) -> int:
    """The context bound the library uses: max_context_len, or max_blocks * block_size if 0."""
    cap = block_tables.shape[1] * block_size
    return cap if max_context_len <= 0 else min(cap, max_context_len)


def alloc_workspace(num_seqs: int, num_heads: int, head_dim: int, capacity: int,
                    partition_size: int = 512, device=None) -> torch.Tensor:
    n = decode_workspace_bytes(num_seqs, num_heads, head_dim, capacity, partition_size)
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
           max_context_len: int = 0, partition_size: int = 512,
           workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None, phases: int = PHASE_ALL) -> torch.Tensor:
    """Paged decode attention; writes and returns ``out`` [S][Hq][d]."""
    NB, Hkv, B, d = k_cache.shape
    S, Hq, dq = q.shape
    if dq != d or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("q, k_cache and v_cache disagree on head_dim / shape")
    if tuple(out.shape) != (S, Hq, d):
        raise ValueError("out must be [num_seqs][num_heads][head_dim]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or tuple(context_lens.shape) != (S,):
        raise ValueError("block_tables must be [num_seqs][max_blocks] and context_lens [num_seqs]")
    dt = k_cache.dtype
    if workspace is None:
        cap = decode_capacity(block_tables, B, max_context_len)
        with _allocating_for(stream):
            workspace = alloc_workspace(S, Hq, d, cap, partition_size, q.device)
    rc = lib.pa_decode_phases(
        _dev(out, "out"), dtype_code(out.dtype), _dev(q, "q", dt), _dev(k_cache, "k_cache", dt),
        _dev(v_cache, "v_cache", dt), _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32), S, Hq, Hkv, d, B, NB,
        block_tables.shape[1], max_context_len, float(scale), partition_size,
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), dtype_code(dt),
        _opt_err(dev_err), _stream_handle(stream), phases)
    _check(rc, "pa_decode")
    return out


def decode_step(out: torch.Tensor, q: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                k_cache: torch.Tensor, v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
                copy_pairs: Optional[torch.Tensor] = None, max_context_len: int = 0, partition_size: int = 512,
                workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One decode step in one call: copy-on-write copies (int64 [n][2]), the
    scatter of key/value [T][Hkv][d] through slot_mapping, and paged decode
    attention; writes and returns ``out`` [S][Hq][d]."""
    NB, Hkv, B, d = k_cache.shape
    S, Hq, dq = q.shape
    T = key.shape[0]
    if dq != d or tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(out.shape) != (S, Hq, d):
        raise ValueError("q / out must be [num_seqs][num_heads][head_dim] over the pool's head_dim")
    if tuple(key.shape) != (T, Hkv, d) or tuple(value.shape) != (T, Hkv, d) or tuple(slot_mapping.shape) != (T,):
        raise ValueError("key/value must be [T][num_kv_heads][head_dim] and slot_mapping [T]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or tuple(context_lens.shape) != (S,):
        raise ValueError("block_tables must be [num_seqs][max_blocks] and context_lens [num_seqs]")
    npairs = 0 if copy_pairs is None else int(copy_pairs.shape[0])
    if npairs and (copy_pairs.dim() != 2 or copy_pairs.shape[1] != 2):
        raise ValueError("copy_pairs must be int64 [n][2]")
    dt = k_cache.dtype
    if workspace is None:
        cap = decode_capacity(block_tables, B, max_context_len)
        with _allocating_for(stream):
            workspace = alloc_workspace(S, Hq, d, cap, partition_size, q.device)
    rc = lib.pa_decode_step(
        _dev(out, "out"), dtype_code(out.dtype), _dev(q, "q", dt), _dev(key, "key", dt) if T else None,
        _dev(value, "value", dt) if T else None, _dev(k_cache, "k_cache", dt), _dev(v_cache, "v_cache", dt),
        _dev(slot_mapping, "slot_mapping", torch.int64) if T else None, T,
        _dev(copy_pairs, "copy_pairs", torch.int64) if npairs else None, npairs,
        _dev(block_tables, "block_tables", torch.int32), _dev(context_lens, "context_lens", torch.int32), S, Hq,
        Hkv, d, B, NB, block_tables.shape[1], max_context_len, float(scale), partition_size,
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), dtype_code(dt), _opt_err(dev_err),
        _stream_handle(stream))
    _check(rc, "pa_decode_step")
    return out


def prefill(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
            block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor, scale: float,
            *, max_context_len: int = 0, partition_size: int = 512,
            workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention of new tokens q [T][Hq][d] (sequence s owns rows
    query_start[s]..query_start[s+1]-1) against the paged context; writes ``out``."""
    NB, Hkv, B, d = k_cache.shape
    T, Hq, dq = q.shape
    S = context_lens.shape[0]
    if dq != d or tuple(out.shape) != (T, Hq, d) or tuple(query_start.shape) != (S + 1,):
        raise ValueError("q/out must be [num_tokens][num_heads][head_dim], query_start [num_seqs + 1]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs][max_blocks]")
    dt = k_cache.dtype
    if workspace is None:
        cap = decode_capacity(block_tables, B, max_context_len)
        n = lib.pa_prefill_workspace_bytes(T, Hq, d, cap, partition_size)
        with _allocating_for(stream):
            workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    rc = lib.pa_prefill(
        _dev(out, "out"), dtype_code(out.dtype), _dev(q, "q", dt), _dev(k_cache, "k_cache", dt),
        _dev(v_cache, "v_cache", dt), _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32), _dev(query_start, "query_start", torch.int32), S, T,
        Hq, Hkv, d, B, NB, block_tables.shape[1], max_context_len, float(scale), partition_size,
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), dtype_code(dt), _opt_err(dev_err),
        _stream_handle(stream))
    _check(rc, "pa_prefill")
    return out


def prefill_uses_tensor_cores(dtype: torch.dtype, num_heads: int, num_kv_heads: int, head_dim: int,
                              block_size: int) -> bool:
    """Whether ``prefill`` serves this shape with the tensor-core (tcgen05) kernel."""
    return bool(lib.pa_prefill_uses_tensor_cores(dtype_code(dtype), num_heads, num_kv_heads, head_dim,
                                                 block_size))


def selftest_bounded_wait(dev_err: torch.Tensor, limit_ns: int = 1_000_000,
                          stream: Optional[torch.cuda.Stream] = None) -> None:
    """Launch the device self-test of the bounded wait: it must OR
    DEVERR_TIMEOUT into dev_err after limit_ns and return."""
    rc = lib.pa_selftest_bounded_wait(_dev(dev_err, "dev_err", torch.int32), int(limit_ns), _stream_handle(stream))
    _check(rc, "pa_selftest_bounded_wait")


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, src_dst_pairs: torch.Tensor,
                dev_err: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy whole blocks src -> dst (int64 [n][2] on the device) in both pools."""
    if tuple(v_cache.shape) != tuple(k_cache.shape) or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must match")
    n = src_dst_pairs.shape[0]
    if src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [num_pairs][2]")
    block_bytes = k_cache[0].numel() * k_cache.element_size()
    rc = lib.pa_copy_blocks(_dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                            _dev(src_dst_pairs, "src_dst_pairs", torch.int64), n, block_bytes,
                            k_cache.shape[0], _opt_err(dev_err), _stream_handle(stream))
    _check(rc, "pa_copy_blocks")


TREE_MAX_WORDS = 8


def alloc_tree_workspace(num_tokens: int, num_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """Workspace of ``tree_decode`` for up to ``num_tokens`` drafted tokens."""
    n = lib.pa_tree_workspace_bytes(num_tokens, num_heads, head_dim)
    if n == 0:
        raise ValueError("invalid arguments for pa_tree_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def tree_uses_tensor_cores(dtype: torch.dtype, block_size: int) -> bool:
    """Whether ``tree_decode`` serves such a pool on the tensor cores (tcgen05)."""
    return bool(lib.pa_tree_uses_tensor_cores(dtype_code(dtype), block_size))


def tree_mask(parents, mask_words: Optional[int] = None) -> torch.Tensor:
    """Mask rows of one tree (int64 [n][mask_words], host): parents[i] is node i's parent, a node
    before it, or negative where it follows the prefix."""
    import numpy as np

    p = np.ascontiguousarray(parents, dtype=np.int32)
    words = max(1, -(-len(p) // 64)) if mask_words is None else int(mask_words)
    mask = np.zeros((len(p), max(words, 1)), dtype=np.int64)
    _check(lib.pa_tree_mask(p.ctypes.data, len(p), words, mask.ctypes.data), "pa_tree_mask")
    return torch.from_numpy(mask)


def tree_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor,
                mask: torch.Tensor, scale: float, *, max_context_len: int = 0,
                workspace: Optional[torch.Tensor] = None, dev_err: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of drafted tokens q [T][Hq][d] (sequence s owns rows query_start[s] ..
    query_start[s+1]-1) against the paged context: each sees its sequence's prefix and the nodes its
    ``mask`` row (int64 [T][words], see ``tree_mask``) names.  Writes and returns ``out``."""
    NB, Hkv, B, d = k_cache.shape
    T, Hq, dq = q.shape
    S = context_lens.shape[0]
    if dq != d or v_cache.shape != k_cache.shape or out.shape != q.shape or tuple(query_start.shape) != (S + 1,):
        raise ValueError("q/out must be [num_tokens][num_heads][head_dim], query_start [num_seqs + 1]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs][max_blocks]")
    if mask.dim() != 2 or mask.shape[0] != T:
        raise ValueError("mask must be [num_tokens][words]")
    dt = k_cache.dtype
    if workspace is None:
        with _allocating_for(stream):
            workspace = alloc_tree_workspace(T, Hq, d, q.device)
    rc = lib.pa_tree_decode(
        _dev(out, "out"), dtype_code(out.dtype), _dev(q, "q", dt), _dev(k_cache, "k_cache", dt),
        _dev(v_cache, "v_cache", dt), _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32), _dev(query_start, "query_start", torch.int32),
        _dev(mask, "mask", torch.int64), mask.shape[1], S, T, Hq, Hkv, d, B, NB, block_tables.shape[1],
        max_context_len, float(scale), _dev(workspace, "workspace", torch.uint8), workspace.numel(), dtype_code(dt),
        _opt_err(dev_err), _stream_handle(stream))
    _check(rc, "pa_tree_decode")
    return out


def alloc_weights_workspace(num_seqs: int, num_heads: int, head_dim: int, capacity: int,
                            partition_size: int = 512, device=None) -> torch.Tensor:
    """Workspace of ``decode_weights`` for contexts up to ``capacity`` tokens."""
    n = lib.pa_decode_weights_workspace_bytes(num_seqs, num_heads, head_dim, capacity, partition_size)
    if n == 0:
        raise ValueError("invalid arguments for pa_decode_weights_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def decode_weights(out: torch.Tensor, weights_out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
                   weights_in: Optional[torch.Tensor] = None, weights_lens: Optional[torch.Tensor] = None,
                   max_context_len: int = 0, partition_size: int = 512, workspace: Optional[torch.Tensor] = None,
                   dev_err: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged decode attention that also adds every cached token's attention weight, summed over the
    query heads of its kv head, to its running total: ``weights_out`` = ``weights_in`` (fp32
    [S][Hkv][stride], or None: zeros; may be ``weights_out``) + the step's weights.  Writes and
    returns ``out`` [S][Hq][d]."""
    NB, Hkv, B, d = k_cache.shape
    S, Hq, dq = q.shape
    if dq != d or v_cache.shape != k_cache.shape or out.shape != q.shape:
        raise ValueError("q / out must be [num_seqs][num_heads][head_dim] over the pool's head_dim")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or tuple(context_lens.shape) != (S,):
        raise ValueError("block_tables must be [num_seqs][max_blocks] and context_lens [num_seqs]")
    if weights_out.dim() != 3 or tuple(weights_out.shape[:2]) != (S, Hkv):
        raise ValueError("weights_out must be [num_seqs][num_kv_heads][stride]")
    if weights_in is not None and weights_in.shape != weights_out.shape:
        raise ValueError("weights_in and weights_out must have the same shape")
    if weights_lens is not None and tuple(weights_lens.shape) != (S,):
        raise ValueError("weights_lens must be [num_seqs]")
    dt = k_cache.dtype
    if workspace is None:
        cap = decode_capacity(block_tables, B, max_context_len)
        with _allocating_for(stream):
            workspace = alloc_weights_workspace(S, Hq, d, cap, partition_size, q.device)
    f32 = torch.float32
    rc = lib.pa_decode_weights(
        _dev(out, "out"), dtype_code(out.dtype), _dev(weights_out, "weights_out", f32),
        None if weights_in is None else _dev(weights_in, "weights_in", f32),
        None if weights_lens is None else _dev(weights_lens, "weights_lens", torch.int32), weights_out.shape[2],
        _dev(q, "q", dt), _dev(k_cache, "k_cache", dt), _dev(v_cache, "v_cache", dt),
        _dev(block_tables, "block_tables", torch.int32), _dev(context_lens, "context_lens", torch.int32), S, Hq, Hkv, d,
        B, NB, block_tables.shape[1], max_context_len, float(scale), partition_size,
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), dtype_code(dt), _opt_err(dev_err),
        _stream_handle(stream))
    _check(rc, "pa_decode_weights")
    return out


def select_tokens(keep: torch.Tensor, keep_lens: torch.Tensor, weights: torch.Tensor, context_lens: torch.Tensor,
                  budgets: torch.Tensor, *, recent: int = 0, dev_err: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Positions to keep of each sequence and kv head: the last ``recent`` ones and those with the
    largest totals (``weights`` fp32 [S][Hkv][stride]) up to ``budgets`` (int32 [S]), ascending, into
    ``keep`` (int32 [S][Hkv][width]) and their number into ``keep_lens`` (int32 [S])."""
    if weights.dim() != 3 or keep.dim() != 3 or keep.shape[:2] != weights.shape[:2]:
        raise ValueError("weights must be [num_seqs][num_kv_heads][stride] and keep [num_seqs][num_kv_heads][width]")
    S, Hkv, stride = weights.shape
    if tuple(keep_lens.shape) != (S,) or tuple(context_lens.shape) != (S,) or tuple(budgets.shape) != (S,):
        raise ValueError("keep_lens, context_lens and budgets must be [num_seqs]")
    i32 = torch.int32
    rc = lib.pa_select_tokens(
        _dev(keep, "keep", i32), _dev(keep_lens, "keep_lens", i32), _dev(weights, "weights", torch.float32),
        _dev(context_lens, "context_lens", i32), _dev(budgets, "budgets", i32), S, Hkv, stride, keep.shape[2],
        int(recent), _opt_err(dev_err), _stream_handle(stream))
    _check(rc, "pa_select_tokens")
    return keep


def compact(k_cache: torch.Tensor, v_cache: torch.Tensor, src_tables: torch.Tensor, dst_tables: torch.Tensor,
            keep: torch.Tensor, keep_lens: torch.Tensor, *, starts: Optional[torch.Tensor] = None,
            weights_in: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
            dev_err: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Move the kept tokens' K, V (and totals) to consecutive positions: position ``keep[s][h][j]``
    (through ``src_tables``) goes to ``starts[s] + j`` (through ``dst_tables``, which may be
    ``src_tables``).  ``keep`` is int32 [S][Hkv][width], or [S][1][width] for the same positions in
    every kv head; ``starts`` None means 0."""
    NB, Hkv, B, d = k_cache.shape
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must match")
    S = keep_lens.shape[0]
    if keep.dim() != 3 or keep.shape[0] != S or keep.shape[1] not in (1, Hkv):
        raise ValueError("keep must be [num_seqs][num_kv_heads or 1][width] and keep_lens [num_seqs]")
    if src_tables.dim() != 2 or dst_tables.dim() != 2 or src_tables.shape[0] != S or dst_tables.shape[0] != S:
        raise ValueError("src_tables and dst_tables must be [num_seqs][max_blocks]")
    if starts is not None and tuple(starts.shape) != (S,):
        raise ValueError("starts must be [num_seqs]")
    if (weights_in is None) != (weights_out is None):
        raise ValueError("weights_in and weights_out come together")
    stride = 0
    if weights_in is not None:
        if weights_in.dim() != 3 or tuple(weights_in.shape[:2]) != (S, Hkv) or weights_in.shape != weights_out.shape:
            raise ValueError("weights_in and weights_out must be [num_seqs][num_kv_heads][stride]")
        stride = weights_in.shape[2]
    i32, f32, dt = torch.int32, torch.float32, k_cache.dtype
    rc = lib.pa_compact(
        _dev(k_cache, "k_cache", dt), _dev(v_cache, "v_cache", dt),
        None if weights_out is None else _dev(weights_out, "weights_out", f32),
        None if weights_in is None else _dev(weights_in, "weights_in", f32), stride,
        _dev(src_tables, "src_tables", i32), _dev(dst_tables, "dst_tables", i32), src_tables.shape[1],
        dst_tables.shape[1], _dev(keep, "keep", i32), keep.shape[1], keep.shape[2],
        None if starts is None else _dev(starts, "starts", i32), _dev(keep_lens, "keep_lens", i32), S, Hkv, d, B, NB,
        dtype_code(dt), _opt_err(dev_err), _stream_handle(stream))
    _check(rc, "pa_compact")


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def decode_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
                   max_context_len: int = 0, partition_size: int = 512,
                   dev_err: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged decode attention for callers that cannot allocate device memory: like
    ``decode`` but with the workspace in a fixed 64 MiB array inside the library
    (shared by all calls on a device; calls that overlap on the GPU race)."""
    NB, Hkv, B, d = k_cache.shape
    S, Hq, _ = q.shape
    dt = k_cache.dtype
    rc = lib.pa_decode_noalloc(
        _dev(out, "out"), dtype_code(out.dtype), _dev(q, "q", dt), _dev(k_cache, "k_cache", dt),
        _dev(v_cache, "v_cache", dt), _dev(block_tables, "block_tables", torch.int32),
        _dev(context_lens, "context_lens", torch.int32), S, Hq, Hkv, d, B, NB, block_tables.shape[1],
        max_context_len, float(scale), partition_size, dtype_code(dt), _opt_err(dev_err),
        _stream_handle(stream))
    _check(rc, "pa_decode_noalloc")
    return out


class NativeBlockManager:
    """Handle on the library's host block manager (``pa_bm_*``): free list, ref
    counts, lazy allocation, fork, copy-on-write planning and, optionally,
    prefix caching by chained block keys.  Host memory only."""

    def __init__(self, num_blocks: int, block_size: int, free_order=None, prefix_cache: bool = False):
        import numpy as np

        self._np = np
        self.block_size = int(block_size)
        order = None
        if free_order is not None:
            self._order = np.ascontiguousarray(free_order, dtype=np.int32)
            order = self._order.ctypes.data
        self._h = lib.pa_bm_create(int(num_blocks), int(block_size), order, int(bool(prefix_cache)))
        if not self._h:
            raise ValueError("pa_bm_create rejected its arguments")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            lib.pa_bm_destroy(h)
            self._h = None

    def add(self, seq_id: int) -> None:
        _check(lib.pa_bm_add_sequence(self._h, seq_id), "pa_bm_add_sequence")

    def fork(self, parent: int, child: int) -> None:
        _check(lib.pa_bm_fork(self._h, parent, child), "pa_bm_fork")

    def free(self, seq_id: int) -> None:
        _check(lib.pa_bm_free(self._h, seq_id), "pa_bm_free")

    def append(self, seq_id: int, tokens):
        """Append tokens (a count, or token ids when prefix caching; ids below zero for the nodes of
        a drafted tree, whose blocks the cache leaves out).  Returns (slots int64 array,
        [(src, dst) copies], tokens served from the cache)."""
        np = self._np
        ids = None
        if isinstance(tokens, int):
            n = tokens
        else:
            ids = np.ascontiguousarray(tokens, dtype=np.int32)
            n = len(ids)
        slots = np.empty(max(n, 1), dtype=np.int64)
        cap = max(n, 1)
        copies = np.empty(2 * cap, dtype=np.int64)
        ncopies, ncached = ctypes.c_int(0), ctypes.c_int(0)
        rc = lib.pa_bm_append(self._h, seq_id, None if ids is None else ids.ctypes.data, n, slots.ctypes.data,
                              copies.ctypes.data, cap, ctypes.byref(ncopies), ctypes.byref(ncached))
        _check(rc, "pa_bm_append")
        pairs = [(int(copies[2 * i]), int(copies[2 * i + 1])) for i in range(ncopies.value)]
        return slots[:n], pairs, ncached.value

    def append_batch(self, seq_ids, tokens, max_copies=None, counts=None):
        """One call for a batch: tokens[k] (a count, or token ids when prefix
        caching) appended to seq_ids[k].  With `counts` given, `tokens` is
        instead one flat array of all the token ids in order (or None without
        prefix caching), as a serving loop holds them.  Returns (slots of all
        new tokens in order, [(src, dst) copies], tokens served from the cache)."""
        np = self._np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        if counts is not None:
            counts = np.ascontiguousarray(counts, dtype=np.int32)
            toks = None if tokens is None else np.ascontiguousarray(tokens, dtype=np.int32)
            if toks is not None and toks.size != int(counts.sum()):
                raise ValueError("tokens must hold sum(counts) token ids")
        elif all(isinstance(t, (int, np.integer)) for t in tokens):
            counts = np.ascontiguousarray(tokens, dtype=np.int32)
            toks = None
        else:
            counts = np.array([len(t) for t in tokens], dtype=np.int32)
            toks = np.ascontiguousarray(np.concatenate([np.asarray(t, dtype=np.int32) for t in tokens])
                                        if len(tokens) else np.zeros(0, dtype=np.int32), dtype=np.int32)
        total = int(counts.sum())
        slots = np.empty(max(total, 1), dtype=np.int64)
        cap = max(total, 1) if max_copies is None else int(max_copies)
        copies = np.empty(2 * max(cap, 1), dtype=np.int64)
        ncopies, ncached = ctypes.c_int(0), ctypes.c_int(0)
        rc = lib.pa_bm_append_batch(self._h, len(ids), ids.ctypes.data, counts.ctypes.data,
                                    None if toks is None else toks.ctypes.data, slots.ctypes.data,
                                    copies.ctypes.data, cap, ctypes.byref(ncopies), ctypes.byref(ncached))
        _check(rc, "pa_bm_append_batch")
        pairs = [(int(copies[2 * i]), int(copies[2 * i + 1])) for i in range(ncopies.value)]
        return slots[:total], pairs, ncached.value

    def compact(self, seq_ids, unchanged, num_tokens, token_ids=None):
        """Bookkeeping of one ``compact`` call: seq_ids[k] keeps num_tokens[k] tokens, the first
        unchanged[k] of them in place.  token_ids (prefix caching): the ids of the others, all
        sequences' in a row, or None if unknown.  Returns the [(src, dst)] block copies to run
        before the moves."""
        np = self._np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        u = np.ascontiguousarray(unchanged, dtype=np.int64)
        n = np.ascontiguousarray(num_tokens, dtype=np.int64)
        if not ids.shape == u.shape == n.shape or ids.ndim != 1:
            raise ValueError("seq_ids, unchanged and num_tokens must be one value per sequence")
        toks = None
        if token_ids is not None:
            toks = np.ascontiguousarray(token_ids, dtype=np.int32)
            if toks.size != int((n - u).sum()):
                raise ValueError("token_ids must hold sum(num_tokens - unchanged) ids")
        copies = np.empty(2 * max(len(ids), 1), dtype=np.int64)
        ncopies = ctypes.c_int(0)
        rc = lib.pa_bm_compact(self._h, len(ids), ids.ctypes.data, u.ctypes.data, n.ctypes.data,
                               None if toks is None else toks.ctypes.data, copies.ctypes.data, ctypes.byref(ncopies))
        _check(rc, "pa_bm_compact")
        return [(int(copies[2 * i]), int(copies[2 * i + 1])) for i in range(ncopies.value)]

    def block_table(self, seq_id: int):
        np = self._np
        nb, nt = ctypes.c_int(0), ctypes.c_int64(0)
        rc = lib.pa_bm_block_table(self._h, seq_id, None, 0, ctypes.byref(nb), ctypes.byref(nt))
        if rc not in (PA_OK, PA_ERR_WORKSPACE):
            _check(rc, "pa_bm_block_table")
        out = np.empty(max(nb.value, 1), dtype=np.int32)
        _check(lib.pa_bm_block_table(self._h, seq_id, out.ctypes.data, len(out), ctypes.byref(nb),
                                     ctypes.byref(nt)), "pa_bm_block_table")
        return [int(b) for b in out[: nb.value]]

    def num_tokens(self, seq_id: int) -> int:
        nb, nt = ctypes.c_int(0), ctypes.c_int64(0)
        lib.pa_bm_block_table(self._h, seq_id, None, 0, ctypes.byref(nb), ctypes.byref(nt))
        return int(nt.value)

    @property
    def num_free(self) -> int:
        return int(lib.pa_bm_num_free(self._h))

    def ref_count(self, block: int) -> int:
        return int(lib.pa_bm_ref_count(self._h, block))
