"""Python binding of the C ABI, one function per entry point, same names.

Argument marshalling only: shapes are read from the tensors, pointers and the
current CUDA stream are passed to ``libpagedattn.so``, and a non-zero status
raises ``PagedAttnError``.  Every step of the computation runs in the
library's kernels; PyTorch provides device memory and streams.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._lib import PA_BF16, PA_FP16, PA_FP8_E4M3, PagedAttnError  # noqa: F401  (re-exported)

_DTYPES = {torch.float16: PA_FP16, torch.bfloat16: PA_BF16}
# E4M3 pools: uint8 codes, or torch's float8_e4m3fn (the same bytes)
_CODE_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}: float16 or bfloat16")
    return _DTYPES[t.dtype]


def _stream_ptr(t: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None:  # the raw handle: building a Stream object costs 2 us a call
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return int(stream.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return int(t.data_ptr())


def _need_codes(t: torch.Tensor, name: str, device: torch.device) -> int:
    """Pointer of an E4M3 pool (uint8 or float8_e4m3fn, contiguous, on `device`)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _CODE_DTYPES:
        raise TypeError(f"{name} must be a uint8 or float8_e4m3fn tensor of E4M3 codes")
    return _need(t, name, t.dtype, device)


def _cuda_device(t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError("paged attention tensors must live on a CUDA device")
    return t.device


def pa_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write key/value [T, Hk, d] into the pools [N, B, Hk, d] at slot_mapping [T] (int64)."""
    dev = _cuda_device(k_cache)
    N, B, Hk, d = k_cache.shape
    T = key.shape[0]
    if key.shape != (T, Hk, d) or value.shape != (T, Hk, d) or v_cache.shape != k_cache.shape:
        raise ValueError("key/value must be [T, Hk, d] matching the pools [N, B, Hk, d]")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    dt = k_cache.dtype
    st = _lib.lib().pa_reshape_and_cache(
        _need(key, "key", dt, dev), _need(value, "value", dt, dev),
        _need(k_cache, "k_cache", dt, dev), _need(v_cache, "v_cache", dt, dev),
        _need(slot_mapping, "slot_mapping", torch.int64, dev), T, N, B, Hk, d, _dtype_code(k_cache),
        _stream_ptr(k_cache, stream))
    _lib.check("pa_reshape_and_cache", st)


def pa_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, block_mapping: torch.Tensor,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy whole blocks: for each row (src, dst) of block_mapping [n, 2] (int64),
    k_cache[dst] = k_cache[src] and v_cache[dst] = v_cache[src]."""
    dev = _cuda_device(k_cache)
    N, B, Hk, d = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if block_mapping.dim() != 2 or block_mapping.shape[1] != 2:
        raise ValueError("block_mapping must be [n, 2]")
    dt = k_cache.dtype
    code = PA_FP8_E4M3 if dt in _CODE_DTYPES else _dtype_code(k_cache)
    st = _lib.lib().pa_copy_blocks(
        _need(k_cache, "k_cache", dt, dev), _need(v_cache, "v_cache", dt, dev),
        _need(block_mapping, "block_mapping", torch.int64, dev), int(block_mapping.shape[0]), N, B, Hk, d,
        code, _stream_ptr(k_cache, stream))
    _lib.check("pa_copy_blocks", st)


def _decode_common(out, q, k_cache, v_cache, block_tables, context_lens, codes: bool = False):
    dev = _cuda_device(q)
    S, H, d = q.shape
    N, B, Hk, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape or out.shape != q.shape:
        raise ValueError("q/out [S, H, d] must match the pools [N, B, Hk, d]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("block_tables must be [S, M] and context_lens [S]")
    dt = q.dtype
    _dtype_code(q)
    if codes:
        pk, pv = _need_codes(k_cache, "k_cache", dev), _need_codes(v_cache, "v_cache", dev)
    else:
        pk, pv = _need(k_cache, "k_cache", dt, dev), _need(v_cache, "v_cache", dt, dev)
    ptrs = (_need(out, "out", dt, dev), _need(q, "q", dt, dev), pk, pv,
            _need(block_tables, "block_tables", torch.int32, dev))
    cl = _need(context_lens, "context_lens", torch.int32, dev)
    return dev, S, H, d, N, B, Hk, int(block_tables.shape[1]), ptrs, cl


def pa_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
              stream: Optional[torch.cuda.Stream] = None) -> None:
    """Single-pass paged decode: out[S, H, d] = attention of q over each sequence's paged KV."""
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl = _decode_common(
        out, q, k_cache, v_cache, block_tables, context_lens)
    st = _lib.lib().pa_decode(po, pq, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N, float(scale), _dtype_code(q),
                              _stream_ptr(q, stream))
    _lib.check("pa_decode", st)


def pa_splitk_workspace_bytes(num_seqs: int, num_heads: int, head_dim: int,
                              max_num_partitions: int) -> int:
    return int(_lib.lib().pa_splitk_workspace_bytes(num_seqs, num_heads, head_dim, max_num_partitions))


def max_num_partitions_for(max_blocks_per_seq: int, block_size: int, partition_size: int) -> int:
    return -(-(max_blocks_per_seq * block_size) // partition_size)


def pa_decode_splitk(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                     partition_size: int, workspace: torch.Tensor,
                     max_num_partitions: Optional[int] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """Split-K paged decode; follow with pa_splitk_reduce on the same stream."""
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl = _decode_common(
        out, q, k_cache, v_cache, block_tables, context_lens)
    P = max_num_partitions or max_num_partitions_for(M, B, partition_size)
    ws = _need(workspace, "workspace", workspace.dtype, dev)
    st = _lib.lib().pa_decode_splitk(po, pq, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N, float(scale),
                                     _dtype_code(q), int(partition_size), int(P), ws,
                                     workspace.numel() * workspace.element_size(),
                                     _stream_ptr(q, stream))
    _lib.check("pa_decode_splitk", st)


def pa_splitk_reduce(out: torch.Tensor, workspace: torch.Tensor, context_lens: torch.Tensor,
                     max_blocks_per_seq: int, block_size: int, partition_size: int,
                     max_num_partitions: Optional[int] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """Merge the partitions of pa_decode_splitk into out[S, H, d]."""
    dev = _cuda_device(out)
    S, H, d = out.shape
    P = max_num_partitions or max_num_partitions_for(max_blocks_per_seq, block_size, partition_size)
    st = _lib.lib().pa_splitk_reduce(
        _need(out, "out", out.dtype, dev), _need(workspace, "workspace", workspace.dtype, dev),
        workspace.numel() * workspace.element_size(), _need(context_lens, "context_lens", torch.int32, dev),
        int(max_blocks_per_seq), int(block_size), S, H, d, int(partition_size), int(P), _dtype_code(out),
        _stream_ptr(out, stream))
    _lib.check("pa_splitk_reduce", st)


def pa_decode_splitk_static(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, scale: float, partition_size: int,
                            stream: Optional[torch.cuda.Stream] = None) -> None:
    """Split-K decode + reduce for callers that cannot allocate device memory:
    the partials go to a fixed array inside the library (at most
    PA_STATIC_SCRATCH_BYTES, 32 MiB).  Calls that overlap on the GPU race on
    that array; the first call on a device should precede any stream capture."""
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl = _decode_common(
        out, q, k_cache, v_cache, block_tables, context_lens)
    st = _lib.lib().pa_decode_splitk_static(po, pq, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N,
                                            float(scale), _dtype_code(q), int(partition_size),
                                            _stream_ptr(q, stream))
    _lib.check("pa_decode_splitk_static", st)


def pa_reshape_and_cache_fp8(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, slot_mapping: torch.Tensor, k_scale: float,
                             v_scale: float, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise key/value [T, Hk, d] (float16 or bfloat16) into the E4M3 pools
    [N, B, Hk, d] (uint8 codes) at slot_mapping [T]: code = E4M3(x / scale)."""
    dev = _cuda_device(k_cache)
    N, B, Hk, d = k_cache.shape
    T = key.shape[0]
    if key.shape != (T, Hk, d) or value.shape != (T, Hk, d) or v_cache.shape != k_cache.shape:
        raise ValueError("key/value must be [T, Hk, d] matching the pools [N, B, Hk, d]")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    dt = key.dtype
    st = _lib.lib().pa_reshape_and_cache_fp8(
        _need(key, "key", dt, dev), _need(value, "value", dt, dev),
        _need_codes(k_cache, "k_cache", dev), _need_codes(v_cache, "v_cache", dev),
        _need(slot_mapping, "slot_mapping", torch.int64, dev), T, N, B, Hk, d, _dtype_code(key),
        float(k_scale), float(v_scale), _stream_ptr(k_cache, stream))
    _lib.check("pa_reshape_and_cache_fp8", st)


def pa_decode_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, k_scale: float,
                  v_scale: float, stream: Optional[torch.cuda.Stream] = None) -> None:
    """pa_decode over E4M3 pools whose values are code * k_scale (K) and code * v_scale (V)."""
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl = _decode_common(
        out, q, k_cache, v_cache, block_tables, context_lens, codes=True)
    st = _lib.lib().pa_decode_fp8(po, pq, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N, float(scale),
                                  _dtype_code(q), float(k_scale), float(v_scale), _stream_ptr(q, stream))
    _lib.check("pa_decode_fp8", st)


def pa_decode_splitk_fp8(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                         k_scale: float, v_scale: float, partition_size: int, workspace: torch.Tensor,
                         max_num_partitions: Optional[int] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """Split-K decode over E4M3 pools; follow with pa_splitk_reduce on the same stream."""
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl = _decode_common(
        out, q, k_cache, v_cache, block_tables, context_lens, codes=True)
    P = max_num_partitions or max_num_partitions_for(M, B, partition_size)
    ws = _need(workspace, "workspace", workspace.dtype, dev)
    st = _lib.lib().pa_decode_splitk_fp8(po, pq, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N, float(scale),
                                         _dtype_code(q), float(k_scale), float(v_scale), int(partition_size),
                                         int(P), ws, workspace.numel() * workspace.element_size(),
                                         _stream_ptr(q, stream))
    _lib.check("pa_decode_splitk_fp8", st)


def pa_decode_prefix_splitk(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                            seqs_per_group: int, prefix_lens: torch.Tensor, partition_size: int,
                            workspace: torch.Tensor, max_num_partitions: Optional[int] = None,
                            k_scale: float = 1.0, v_scale: float = 1.0,
                            stream: Optional[torch.cuda.Stream] = None) -> None:
    """Split-K decode that reads each group's shared prompt blocks once: sequences
    [j*seqs_per_group, (j+1)*seqs_per_group) share their first prefix_lens[j] tokens
    (int32 [ceil(S / seqs_per_group)], multiples of partition_size).  E4M3 pools
    (uint8 / float8_e4m3fn) take k_scale and v_scale.  Follow with pa_splitk_reduce."""
    codes = k_cache.dtype in _CODE_DTYPES
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl = _decode_common(
        out, q, k_cache, v_cache, block_tables, context_lens, codes=codes)
    ngroups = -(-S // int(seqs_per_group)) if seqs_per_group > 0 else 0
    if prefix_lens.shape != (ngroups,):
        raise ValueError(f"prefix_lens must be [{ngroups}] (one entry per group)")
    P = max_num_partitions or max_num_partitions_for(M, B, partition_size)
    ws = _need(workspace, "workspace", workspace.dtype, dev)
    dt = _dtype_code(q)
    kv = PA_FP8_E4M3 if codes else dt
    st = _lib.lib().pa_decode_prefix_splitk(
        po, pq, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N, float(scale), dt, kv, float(k_scale), float(v_scale),
        int(seqs_per_group), _need(prefix_lens, "prefix_lens", torch.int32, dev), int(partition_size), int(P), ws,
        workspace.numel() * workspace.element_size(), _stream_ptr(q, stream))
    _lib.check("pa_decode_prefix_splitk", st)


def _append_common(out, q, key, value, k_cache, v_cache, block_tables, context_lens):
    codes = k_cache.dtype in _CODE_DTYPES
    dev, S, H, d, N, B, Hk, M, ptrs, pcl = _decode_common(out, q, k_cache, v_cache, block_tables, context_lens,
                                                          codes=codes)
    if key.shape != (S, Hk, d) or value.shape != (S, Hk, d):
        raise ValueError("key/value must be [S, Hk, d]: one new token per sequence")
    pkey, pval = _need(key, "key", q.dtype, dev), _need(value, "value", q.dtype, dev)
    dt = _dtype_code(q)
    return dev, S, H, d, N, B, Hk, M, ptrs, pcl, pkey, pval, dt, (PA_FP8_E4M3 if codes else dt)


def pa_append_and_decode(out: torch.Tensor, q: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                         k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                         context_lens: torch.Tensor, scale: float, k_scale: float = 1.0, v_scale: float = 1.0,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """One decode step in one launch: key/value [S, Hk, d] (one new token per sequence) go
    into the pools at position context_lens[s] - 1, then out = pa_decode over the whole
    context.  E4M3 pools (uint8 / float8_e4m3fn) take k_scale and v_scale."""
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl, pkey, pval, dt, kv = _append_common(
        out, q, key, value, k_cache, v_cache, block_tables, context_lens)
    st = _lib.lib().pa_append_and_decode(po, pq, pkey, pval, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N, float(scale),
                                         dt, kv, float(k_scale), float(v_scale), _stream_ptr(q, stream))
    _lib.check("pa_append_and_decode", st)


def pa_append_and_decode_splitk(out: torch.Tensor, q: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                                k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                                context_lens: torch.Tensor, scale: float, partition_size: int,
                                workspace: torch.Tensor, max_num_partitions: Optional[int] = None,
                                k_scale: float = 1.0, v_scale: float = 1.0,
                                stream: Optional[torch.cuda.Stream] = None) -> None:
    """pa_append_and_decode with the split-K partitions; follow with pa_splitk_reduce."""
    dev, S, H, d, N, B, Hk, M, (po, pq, pk, pv, pbt), pcl, pkey, pval, dt, kv = _append_common(
        out, q, key, value, k_cache, v_cache, block_tables, context_lens)
    P = max_num_partitions or max_num_partitions_for(M, B, partition_size)
    ws = _need(workspace, "workspace", workspace.dtype, dev)
    st = _lib.lib().pa_append_and_decode_splitk(
        po, pq, pkey, pval, pk, pv, pbt, M, pcl, S, H, Hk, d, B, N, float(scale), dt, kv, float(k_scale),
        float(v_scale), int(partition_size), int(P), ws, workspace.numel() * workspace.element_size(),
        _stream_ptr(q, stream))
    _lib.check("pa_append_and_decode_splitk", st)


def pa_prefill(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
               block_tables: torch.Tensor, context_lens: torch.Tensor, query_start_loc: torch.Tensor,
               max_query_len: int, scale: float, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Paged prefill: q/out [rows, H, d]; sequence s owns rows query_start_loc[s] ..
    query_start_loc[s+1] (its last positions) and each row attends causally."""
    dev = _cuda_device(q)
    R, H, d = q.shape
    N, B, Hk, d2 = k_cache.shape
    S = int(context_lens.shape[0])
    if d2 != d or v_cache.shape != k_cache.shape or out.shape != q.shape:
        raise ValueError("q/out [rows, H, d] must match the pools [N, B, Hk, d]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or query_start_loc.shape != (S + 1,):
        raise ValueError("block_tables must be [S, M] and query_start_loc [S + 1]")
    dt = q.dtype
    st = _lib.lib().pa_prefill(
        _need(out, "out", dt, dev), _need(q, "q", dt, dev), _need(k_cache, "k_cache", dt, dev),
        _need(v_cache, "v_cache", dt, dev), _need(block_tables, "block_tables", torch.int32, dev),
        int(block_tables.shape[1]), _need(context_lens, "context_lens", torch.int32, dev),
        _need(query_start_loc, "query_start_loc", torch.int32, dev), S, R, int(max_query_len), H, Hk, d, B, N,
        float(scale), _dtype_code(q), _stream_ptr(q, stream))
    _lib.check("pa_prefill", st)


# ---------------------------------------------------------------------------
# Block-scaled E4M3 pools and block-sparse decode.  A small decode step is paced
# by the host, so each call first goes the short way through csrc/py_fast.cpp,
# which reads the tensors in C++ and launches when everything is as wanted.  When
# it is not (or the tensors' device is not current), nothing has been launched and
# the call goes on below, where each check has its message.
# ---------------------------------------------------------------------------
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _ptr(t: torch.Tensor, name: str, dtype: torch.dtype, index: int) -> int:
    """Pointer of a contiguous tensor of `dtype` on CUDA device `index`."""
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return _need(t, name, dtype, torch.device("cuda", index))  # raises, with the reason


def _ptr_codes(t: torch.Tensor, name: str, index: int) -> int:
    if t.dtype not in _CODE_DTYPES:
        raise TypeError(f"{name} must be a uint8 or float8_e4m3fn tensor of E4M3 codes")
    return _ptr(t, name, t.dtype, index)


def _cuda_index(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("paged attention tensors must live on a CUDA device")
    return t.get_device()


def _run(fn, name: str, index: int, stream: Optional[torch.cuda.Stream], args: tuple) -> None:
    """Call a launching entry point with its arguments and the stream, the tensors' device current."""
    sp = torch._C._cuda_getCurrentRawStream(index) if stream is None else int(stream.cuda_stream)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, sp)
    else:
        with torch.cuda.device(index):
            st = fn(*args, sp)
    if st:
        _lib.check(name, st)


def _check_scales(k_scales: torch.Tensor, v_scales: torch.Tensor, N: int, Hk: int) -> None:
    if k_scales.shape != (N, Hk) or v_scales.shape != (N, Hk):
        raise ValueError(f"k_scales and v_scales must be [N, Hk] = [{N}, {Hk}], one scale per block and KV head")


def _check_bounds(key_bounds: torch.Tensor, bound_exps: torch.Tensor, Hk: int, d: int) -> int:
    N = key_bounds.shape[0]
    if key_bounds.shape != (N, Hk, 2, d) or bound_exps.shape != (N, Hk):
        raise ValueError(f"key_bounds must be [N, Hk, 2, d] and bound_exps [N, Hk] with Hk = {Hk}, d = {d}")
    return N


def pa_reshape_and_cache_fp8_block(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                                   slot_mapping: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise key/value [T, Hk, d] (float16 or bfloat16) into the E4M3 pools [N, B, Hk, d]
    at slot_mapping [T], with one scale per (block, KV head) in k_scales / v_scales [N, Hk]
    (float32) taken from the data and grown as a block fills.  The tokens of one block
    stand next to each other in slot_mapping."""
    if k_cache.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().write(key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping, dev, sp):
            return
    i = _cuda_index(k_cache)
    shape = k_cache.shape
    N, B, Hk, d = shape
    T = key.shape[0]
    if key.shape != (T, Hk, d) or value.shape != (T, Hk, d) or v_cache.shape != shape:
        raise ValueError("key/value must be [T, Hk, d] matching the pools [N, B, Hk, d]")
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    _check_scales(k_scales, v_scales, N, Hk)
    dt = key.dtype
    _run(_lib.lib().pa_reshape_and_cache_fp8_block, "pa_reshape_and_cache_fp8_block", i, stream,
         (_ptr(key, "key", dt, i), _ptr(value, "value", dt, i), _ptr_codes(k_cache, "k_cache", i),
          _ptr_codes(v_cache, "v_cache", i), _ptr(k_scales, "k_scales", torch.float32, i),
          _ptr(v_scales, "v_scales", torch.float32, i), _ptr(slot_mapping, "slot_mapping", torch.int64, i), T, N, B,
          Hk, d, _dtype_code(key)))


def _block_decode_args(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale):
    i = _cuda_index(q)
    qs, ks = q.shape, k_cache.shape
    S, H, d = qs
    N, B, Hk, d2 = ks
    if d2 != d or v_cache.shape != ks or out.shape != qs:
        raise ValueError("q/out [S, H, d] must match the pools [N, B, Hk, d]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("block_tables must be [S, M] and context_lens [S]")
    _check_scales(k_scales, v_scales, N, Hk)
    dt = q.dtype
    return i, S, H, d, B, block_tables.shape[1], (
        _ptr(out, "out", dt, i), _ptr(q, "q", dt, i), _ptr_codes(k_cache, "k_cache", i),
        _ptr_codes(v_cache, "v_cache", i), _ptr(k_scales, "k_scales", torch.float32, i),
        _ptr(v_scales, "v_scales", torch.float32, i), _ptr(block_tables, "block_tables", torch.int32, i),
        block_tables.shape[1], _ptr(context_lens, "context_lens", torch.int32, i), S, H, Hk, d, B, N, float(scale),
        _dtype_code(q))


def pa_decode_fp8_block(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, scale: float,
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """pa_decode over block-scaled E4M3 pools: values are code * k_scales[block, head] (K) and
    code * v_scales[block, head] (V); q and out are float16 or bfloat16."""
    if q.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().decode(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, dev,
                              sp):
            return
    i, _, _, _, _, _, args = _block_decode_args(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                                                scale)
    _run(_lib.lib().pa_decode_fp8_block, "pa_decode_fp8_block", i, stream, args)


def pa_decode_splitk_fp8_block(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                               context_lens: torch.Tensor, scale: float, partition_size: int,
                               workspace: torch.Tensor, max_num_partitions: Optional[int] = None,
                               stream: Optional[torch.cuda.Stream] = None) -> None:
    """Split-K decode over block-scaled pools; follow with pa_splitk_reduce on the same stream."""
    if q.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        P = max_num_partitions or max_num_partitions_for(block_tables.shape[-1], k_cache.shape[1], partition_size)
        if _lib.fast().splitk(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale,
                              partition_size, P, workspace, dev, sp):
            return
    i, _, _, _, B, M, args = _block_decode_args(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                                                scale)
    P = max_num_partitions or max_num_partitions_for(M, B, partition_size)
    _run(_lib.lib().pa_decode_splitk_fp8_block, "pa_decode_splitk_fp8_block", i, stream,
         args + (int(partition_size), int(P), _ptr(workspace, "workspace", workspace.dtype, i),
                 workspace.numel() * workspace.element_size()))


def pa_prefill_fp8_block(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                         context_lens: torch.Tensor, query_start_loc: torch.Tensor, max_query_len: int,
                         scale: float, stream: Optional[torch.cuda.Stream] = None) -> None:
    """pa_prefill over block-scaled E4M3 pools (k_scales / v_scales [N, Hk])."""
    if q.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().prefill(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                               query_start_loc, max_query_len, scale, dev, sp):
            return
    i = _cuda_index(q)
    qs, ks = q.shape, k_cache.shape
    R, H, d = qs
    N, B, Hk, d2 = ks
    S = context_lens.shape[0]
    if d2 != d or v_cache.shape != ks or out.shape != qs:
        raise ValueError("q/out [rows, H, d] must match the pools [N, B, Hk, d]")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or query_start_loc.shape != (S + 1,):
        raise ValueError("block_tables must be [S, M] and query_start_loc [S + 1]")
    _check_scales(k_scales, v_scales, N, Hk)
    dt = q.dtype
    _run(_lib.lib().pa_prefill_fp8_block, "pa_prefill_fp8_block", i, stream,
         (_ptr(out, "out", dt, i), _ptr(q, "q", dt, i), _ptr_codes(k_cache, "k_cache", i),
          _ptr_codes(v_cache, "v_cache", i), _ptr(k_scales, "k_scales", torch.float32, i),
          _ptr(v_scales, "v_scales", torch.float32, i), _ptr(block_tables, "block_tables", torch.int32, i),
          block_tables.shape[1], _ptr(context_lens, "context_lens", torch.int32, i),
          _ptr(query_start_loc, "query_start_loc", torch.int32, i), S, R, int(max_query_len), H, Hk, d, B, N,
          float(scale), _dtype_code(q)))


def pa_update_key_bounds(key: torch.Tensor, key_bounds: torch.Tensor, bound_exps: torch.Tensor,
                         slot_mapping: torch.Tensor, block_size: int,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """Fold key [T, Hk, d] into the bounds of the blocks named by slot_mapping [T]: key_bounds
    [N, Hk, 2, d] (int8 lo, hi) and bound_exps [N, Hk] (int32), lo * 2^e <= k <= hi * 2^e.
    The tokens of one block stand next to each other in slot_mapping."""
    if key_bounds.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().bounds(key, key_bounds, bound_exps, slot_mapping, block_size, dev, sp):
            return
    i = _cuda_index(key_bounds)
    T, Hk, d = key.shape
    N = _check_bounds(key_bounds, bound_exps, Hk, d)
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must be [T]")
    _run(_lib.lib().pa_update_key_bounds, "pa_update_key_bounds", i, stream,
         (_ptr(key, "key", key.dtype, i), _ptr(key_bounds, "key_bounds", torch.int8, i),
          _ptr(bound_exps, "bound_exps", torch.int32, i), _ptr(slot_mapping, "slot_mapping", torch.int64, i), T, N,
          int(block_size), Hk, d, _dtype_code(key)))


def pa_select_workspace_bytes(num_seqs: int, num_kv_heads: int, max_blocks_per_seq: int) -> int:
    return int(_lib.lib().pa_select_workspace_bytes(num_seqs, num_kv_heads, max_blocks_per_seq))


def alloc_select_workspace(num_seqs: int, num_kv_heads: int, max_blocks_per_seq: int, device) -> torch.Tensor:
    """A float32 device buffer of the size pa_select_workspace_bytes states."""
    nbytes = pa_select_workspace_bytes(num_seqs, num_kv_heads, max_blocks_per_seq)
    return torch.empty(max(1, nbytes // 4), dtype=torch.float32, device=device)


def pa_select_blocks(sel_tables: torch.Tensor, sel_lens: torch.Tensor, q: torch.Tensor, key_bounds: torch.Tensor,
                     bound_exps: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                     block_size: int, num_first: int, num_last: int, workspace: torch.Tensor,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """Choose the blocks that each (sequence, KV head) reads: the first num_first, the last
    num_last and the best by the bounds of their keys, max_selected in all.  Writes
    sel_tables [S, Hk, max_selected] (physical ids in position order, then -1) and
    sel_lens [S, Hk] (tokens), both int32."""
    if q.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().select(sel_tables, sel_lens, q, key_bounds, bound_exps, block_tables, context_lens, block_size,
                              num_first, num_last, workspace, dev, sp):
            return
    i = _cuda_index(q)
    S, H, d = q.shape
    if sel_tables.dim() != 3 or sel_tables.shape[0] != S:
        raise ValueError("sel_tables must be [S, Hk, max_selected]")
    _, Hk, K = sel_tables.shape
    if sel_lens.shape != (S, Hk):
        raise ValueError("sel_lens must be [S, Hk]")
    N = _check_bounds(key_bounds, bound_exps, Hk, d)
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("block_tables must be [S, M] and context_lens [S]")
    _run(_lib.lib().pa_select_blocks, "pa_select_blocks", i, stream,
         (_ptr(sel_tables, "sel_tables", torch.int32, i), _ptr(sel_lens, "sel_lens", torch.int32, i),
          _ptr(q, "q", q.dtype, i), _ptr(key_bounds, "key_bounds", torch.int8, i),
          _ptr(bound_exps, "bound_exps", torch.int32, i), _ptr(block_tables, "block_tables", torch.int32, i),
          block_tables.shape[1], _ptr(context_lens, "context_lens", torch.int32, i), S, H, Hk, d, int(block_size), N, K,
          int(num_first), int(num_last), _dtype_code(q), _ptr(workspace, "workspace", workspace.dtype, i),
          workspace.numel() * workspace.element_size()))


def pa_decode_sparse(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     sel_tables: torch.Tensor, sel_lens: torch.Tensor, scale: float,
                     k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """Decode with a block table per (sequence, KV head): sel_tables [S, Hk, max_selected] and
    sel_lens [S, Hk] (pa_select_blocks writes them).  16-bit pools of the query type, or
    block-scaled E4M3 pools with k_scales and v_scales [N, Hk]."""
    if q.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().sparse(out, q, k_cache, v_cache, sel_tables, sel_lens, scale, k_scales, v_scales, dev, sp):
            return
    i = _cuda_index(q)
    qs, ks = q.shape, k_cache.shape
    S, H, d = qs
    N, B, Hk, d2 = ks
    if d2 != d or v_cache.shape != ks or out.shape != qs:
        raise ValueError("q/out [S, H, d] must match the pools [N, B, Hk, d]")
    if sel_tables.dim() != 3 or sel_tables.shape[:2] != (S, Hk) or sel_lens.shape != (S, Hk):
        raise ValueError("sel_tables must be [S, Hk, max_selected] and sel_lens [S, Hk]")
    dt = q.dtype
    code = _dtype_code(q)
    if k_cache.dtype in _CODE_DTYPES:
        if k_scales is None or v_scales is None:
            raise ValueError("E4M3 pools need k_scales and v_scales [N, Hk]")
        _check_scales(k_scales, v_scales, N, Hk)
        pools = (_ptr_codes(k_cache, "k_cache", i), _ptr_codes(v_cache, "v_cache", i),
                 _ptr(k_scales, "k_scales", torch.float32, i), _ptr(v_scales, "v_scales", torch.float32, i))
        kv = PA_FP8_E4M3
    else:
        if k_scales is not None or v_scales is not None:
            raise ValueError("16-bit pools take no scales")
        pools = (_ptr(k_cache, "k_cache", dt, i), _ptr(v_cache, "v_cache", dt, i), None, None)
        kv = code
    _run(_lib.lib().pa_decode_sparse, "pa_decode_sparse", i, stream,
         (_ptr(out, "out", dt, i), _ptr(q, "q", dt, i)) + pools +
         (_ptr(sel_tables, "sel_tables", torch.int32, i), sel_tables.shape[2],
          _ptr(sel_lens, "sel_lens", torch.int32, i), S, H, Hk, d, B, N, float(scale), code, kv))


# ---------------------------------------------------------------------------
# Whole prompts in packed rows, and the sequences' blocks on the device.
# ---------------------------------------------------------------------------
def _ptr_rows(t: torch.Tensor, name: str, dtype: torch.dtype, index: int):
    """Pointer and row stride (elements) of a [rows, heads, d] tensor whose rows are contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    rows, heads, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"the heads of one token of {name} must be contiguous")
    return t.data_ptr(), t.stride(0) if rows > 1 else heads * d


def pa_prefill_packed(out: torch.Tensor, q: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                      query_start_loc: torch.Tensor, max_query_len: int, scale: float,
                      k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                      slot_mapping: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Causal attention over whole prompts: q [rows, H, d], key and value [rows, Hk, d] (rows
    of any stride: parts of one projection's output will do), sequence s owning the rows
    query_start_loc[s] .. query_start_loc[s+1].  With k_cache, v_cache [N, B, Hk, d] and
    slot_mapping [rows] (int64) the key and value rows go into the pools as well."""
    if q.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().packed(out, q, key, value, query_start_loc, max_query_len, scale, k_cache, v_cache, slot_mapping, dev, sp):
            return
    i = _cuda_index(q)
    R, H, d = q.shape
    Hk = key.shape[1] if key.dim() == 3 else 0
    if out.shape != q.shape or key.shape != (R, Hk, d) or value.shape != key.shape:
        raise ValueError("q/out must be [rows, H, d] and key/value [rows, Hk, d]")
    if query_start_loc.dim() != 1 or query_start_loc.shape[0] < 1:
        raise ValueError("query_start_loc must be [S + 1]")
    S = query_start_loc.shape[0] - 1
    dt = q.dtype
    code = _dtype_code(q)
    N = B = 0
    pools = (None, None, None)
    if k_cache is not None or v_cache is not None or slot_mapping is not None:
        if k_cache is None or v_cache is None or slot_mapping is None:
            raise ValueError("k_cache, v_cache and slot_mapping are given together or not at all")
        if k_cache.dim() != 4 or k_cache.shape[2:] != (Hk, d) or v_cache.shape != k_cache.shape:
            raise ValueError(f"k_cache and v_cache must be [N, B, Hk, d] with Hk = {Hk}, d = {d}")
        if slot_mapping.shape != (R,):
            raise ValueError("slot_mapping must be [rows]")
        N, B = k_cache.shape[:2]
        pools = (_ptr(k_cache, "k_cache", dt, i), _ptr(v_cache, "v_cache", dt, i),
                 _ptr(slot_mapping, "slot_mapping", torch.int64, i))
    _run(_lib.lib().pa_prefill_packed, "pa_prefill_packed", i, stream,
         (_ptr(out, "out", dt, i), *_ptr_rows(q, "q", dt, i), *_ptr_rows(key, "key", dt, i),
          *_ptr_rows(value, "value", dt, i), *pools, _ptr(query_start_loc, "query_start_loc", torch.int32, i), S, R,
          int(max_query_len), H, Hk, d, B, N, float(scale), code))


def pa_sequence_workspace_bytes(num_blocks: int) -> int:
    return int(_lib.lib().pa_sequence_workspace_bytes(num_blocks))


def alloc_sequence_workspace(num_blocks: int, device) -> torch.Tensor:
    """An int32 device buffer of the size pa_sequence_workspace_bytes states."""
    return torch.empty(max(1, pa_sequence_workspace_bytes(num_blocks) // 4), dtype=torch.int32, device=device)


def _sequence_args(block_tables, context_lens, ref_counts):
    """Device index, S, M, N and the pointers of the sequences' tables, lengths and counts."""
    i = _cuda_index(block_tables)
    if block_tables.dim() != 2 or context_lens.shape != (block_tables.shape[0],):
        raise ValueError("block_tables must be [S, M] and context_lens [S]")
    if ref_counts.dim() != 1:
        raise ValueError("ref_counts must be [N]")
    S, M = block_tables.shape
    return i, S, M, ref_counts.shape[0], (_ptr(block_tables, "block_tables", torch.int32, i), M,
                                          _ptr(context_lens, "context_lens", torch.int32, i),
                                          _ptr(ref_counts, "ref_counts", torch.int32, i))


def pa_extend_sequences(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_counts: torch.Tensor,
                        query_start_loc: torch.Tensor, slot_mapping: torch.Tensor, block_copies: torch.Tensor,
                        left: torch.Tensor, block_size: int, workspace: torch.Tensor,
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """Make room for query_start_loc[s+1] - query_start_loc[s] new tokens of each sequence: free
    blocks (ref_counts [N] == 0) go into block_tables [S, M] and context_lens [S] grows.  Writes
    the tokens' slots (slot_mapping, int64), the copies that shared last blocks need
    (block_copies [S, 2], int64) and left [2] (free blocks, refused sequences)."""
    if block_tables.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().extend(block_tables, context_lens, ref_counts, query_start_loc, slot_mapping, block_copies, left,
                              block_size, workspace, dev, sp):
            return
    i, S, M, N, head = _sequence_args(block_tables, context_lens, ref_counts)
    if query_start_loc.shape != (S + 1,):
        raise ValueError("query_start_loc must be [S + 1]")
    if slot_mapping.dim() != 1 or block_copies.shape != (S, 2) or left.shape != (2,):
        raise ValueError("slot_mapping must be [tokens], block_copies [S, 2] and left [2]")
    _run(_lib.lib().pa_extend_sequences, "pa_extend_sequences", i, stream,
         head + (_ptr(query_start_loc, "query_start_loc", torch.int32, i),
                 _ptr(slot_mapping, "slot_mapping", torch.int64, i), _ptr(block_copies, "block_copies", torch.int64, i),
                 _ptr(left, "left", torch.int32, i), S, slot_mapping.shape[0], N, int(block_size),
                 _ptr(workspace, "workspace", workspace.dtype, i), workspace.numel() * workspace.element_size()))


def pa_truncate_sequences(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_counts: torch.Tensor,
                          new_lens: torch.Tensor, block_size: int,
                          stream: Optional[torch.cuda.Stream] = None) -> None:
    """Cut each sequence with 0 <= new_lens[s] < context_lens[s] to new_lens[s] tokens (0: free it)
    and give its blocks back."""
    if block_tables.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().truncate(block_tables, context_lens, ref_counts, new_lens, block_size, dev, sp):
            return
    i, S, M, N, head = _sequence_args(block_tables, context_lens, ref_counts)
    if new_lens.shape != (S,):
        raise ValueError("new_lens must be [S]")
    _run(_lib.lib().pa_truncate_sequences, "pa_truncate_sequences", i, stream,
         head + (_ptr(new_lens, "new_lens", torch.int32, i), S, N, int(block_size)))


def pa_fork_sequences(block_tables: torch.Tensor, context_lens: torch.Tensor, ref_counts: torch.Tensor,
                      fork_from: torch.Tensor, block_size: int, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Each empty sequence with fork_from[s] >= 0 becomes a copy of that sequence and shares its blocks."""
    if block_tables.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().fork(block_tables, context_lens, ref_counts, fork_from, block_size, dev, sp):
            return
    i, S, M, N, head = _sequence_args(block_tables, context_lens, ref_counts)
    if fork_from.shape != (S,):
        raise ValueError("fork_from must be [S]")
    _run(_lib.lib().pa_fork_sequences, "pa_fork_sequences", i, stream,
         head + (_ptr(fork_from, "fork_from", torch.int32, i), S, N, int(block_size)))


def pa_compact_blocks(moves: torch.Tensor, num_moves: torch.Tensor, block_tables: torch.Tensor,
                      context_lens: torch.Tensor, ref_counts: torch.Tensor, tables_out: torch.Tensor,
                      counts_out: torch.Tensor, block_size: int, workspace: torch.Tensor,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Plan at most len(moves) moves of the highest used blocks to the lowest free ones: moves
    [max, 2] (int64), num_moves [1] (int32), and the tables and counts after them (tables_out,
    counts_out: the inputs themselves, or others).  Follow with pa_copy_layer_blocks."""
    if block_tables.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().compact(moves, num_moves, block_tables, context_lens, ref_counts, tables_out, counts_out,
                               block_size, workspace, dev, sp):
            return
    i, S, M, N, (tables, _, lens, counts) = _sequence_args(block_tables, context_lens, ref_counts)
    if moves.dim() != 2 or moves.shape[1] != 2 or num_moves.shape != (1,):
        raise ValueError("moves must be [max_moves, 2] and num_moves [1]")
    if tables_out.shape != block_tables.shape or counts_out.shape != ref_counts.shape:
        raise ValueError("tables_out must be [S, M] and counts_out [N]")
    _run(_lib.lib().pa_compact_blocks, "pa_compact_blocks", i, stream,
         (_ptr(moves, "moves", torch.int64, i), moves.shape[0], _ptr(num_moves, "num_moves", torch.int32, i), tables, M,
          lens, counts, _ptr(tables_out, "tables_out", torch.int32, i), _ptr(counts_out, "counts_out", torch.int32, i), S,
          N, int(block_size), _ptr(workspace, "workspace", workspace.dtype, i),
          workspace.numel() * workspace.element_size()))


def pa_copy_layer_blocks(pools: torch.Tensor, block_mapping: torch.Tensor,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """For each row (src, dst) of block_mapping [n, 2] (int64) and each layer l of pools [L, N, ...]
    (any type; a layer's blocks contiguous): pools[l, dst] = pools[l, src]."""
    if pools.is_cuda:
        dev = _get_device()
        sp = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _lib.fast().copy_layers(pools, block_mapping, dev, sp):
            return
    i = _cuda_index(pools)
    if pools.dim() < 3:
        raise ValueError("pools must be [L, N, ...]: the pools of L layers")
    if block_mapping.dim() != 2 or block_mapping.shape[1] != 2:
        raise ValueError("block_mapping must be [n, 2]")
    L, N = pools.shape[:2]
    if L == 0 or pools.numel() == 0:
        return
    if not pools[0].is_contiguous():
        raise ValueError("the blocks of one layer must be contiguous")
    width = pools.element_size()
    _run(_lib.lib().pa_copy_layer_blocks, "pa_copy_layer_blocks", i, stream,
         (pools.data_ptr(), pools.stride(0) * width, L, pools.numel() // (L * N) * width,
          _ptr(block_mapping, "block_mapping", torch.int64, i), block_mapping.shape[0], N))


def pa_selftest_wait(device=None, limit_us: int = 20000,
                     stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Run the library's bounded-wait self-test on `device` (default: the current CUDA
    device) and return {"gave_up", "completed", "waited_us"} once it has finished."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.type != "cuda":
        raise ValueError("the self-test runs on a CUDA device")
    res = torch.full((3,), -1, dtype=torch.int32, device=dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    st = _lib.lib().pa_selftest_wait(int(res.data_ptr()), int(limit_us), int(s.cuda_stream))
    _lib.check("pa_selftest_wait", st)
    s.synchronize()
    r = res.cpu().tolist()
    return {"gave_up": r[0] == 1, "completed": r[1] == 1, "waited_us": r[2]}


def pa_status_string(status: int) -> str:
    return _lib.status_name(status)


def pa_last_error() -> str:
    return _lib.last_error()


def alloc_splitk_workspace(num_seqs: int, num_heads: int, head_dim: int, max_num_partitions: int,
                           device) -> torch.Tensor:
    """A float32 device buffer of the size pa_splitk_workspace_bytes states."""
    nbytes = pa_splitk_workspace_bytes(num_seqs, num_heads, head_dim, max_num_partitions)
    return torch.empty(max(1, nbytes // 4), dtype=torch.float32, device=device)
