"""GB300 (sm_103a) multi-head latent attention decode over a paged latent KV cache.

A thin Python binding over the C ABI of ``libmla_decode.so``
(``include/mla_decode.h``).  The functions here only marshal torch tensors into
pointers and sizes; every step of the computation runs in the library's CUDA
kernels.  If the library is missing they raise; there is no fallback.

Entry points (same names as the C ABI):
  mla_decode_paged      bf16 paged cache
  mla_decode_paged_fp8  e4m3 latent cache with one fp32 scale per row, e4m3 weights
  mla_decode_paged_fp4  e2m1 latent cache with one power-of-two scale per 32 values
  mla_decode_sparse     attention restricted to given physical cache rows
  mla_cache_append      new latent rows into a bf16, e4m3 or e2m1 cache (RMSNorm, RoPE, codes); RoPE on q
  mla_branch_prologue   RoPE on q and the new cache rows, RMSNorm of their latent part
  mla_prefill_paged     many query tokens a request, expanded form (also _fp8, _fp4)
  mla_indexer_fp8       top-k cache rows per query token by FP8 index scores (sparse input)
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _lib
from ._lib import (MLA_FLAG_DEBUG_CHECKS, MLA_FLAG_KERNEL_TIMING, MLA_FLAG_FOLD_PAIRS, MLA_FLAG_PER_TOKEN,
                   MLA_CACHE_BF16, MLA_CACHE_E2M1, MLA_CACHE_E4M3, MLA_MASK_CAUSAL, MLA_MASK_NULL,
                   MLA_MASK_SLIDING_WINDOW_CAUSAL, MlaDims, MlaError, MlaOpts, kernel_times)

__all__ = ["mla_decode_paged", "mla_decode_paged_fp8", "mla_decode_paged_fp4", "mla_decode_sparse",
           "mla_branch_prologue", "mla_cache_append", "mla_cache_row_bytes", "mla_indexer_fp8",
           "mla_prefill_paged", "mla_prefill_paged_fp8", "mla_prefill_paged_fp4", "mla_prefill_workspace_size",
           "MLA_CACHE_BF16", "MLA_CACHE_E4M3", "MLA_CACHE_E2M1",
           "mla_decode_workspace_size", "MlaDims", "MlaOpts", "MlaError", "MLA_MASK_NULL",
           "MLA_MASK_CAUSAL", "MLA_MASK_SLIDING_WINDOW_CAUSAL", "library_path", "kernel_times"]


def library_path() -> str:
    return _lib.LIB


def _ptr(t: Optional[torch.Tensor], name: str, dtypes=None, device=None):
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and (dtypes is None or t.dtype in dtypes) and t.is_cuda and \
            t.is_contiguous() and (device is None or t.device == device):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.data_ptr()


def _opts(mask, window, scale, num_splits, debug, timing=False, fold_pairs=None) -> MlaOpts:
    # fold_pairs: None = the library's choice, True / False = force pairs / one token at a time
    walk = 0 if fold_pairs is None else (MLA_FLAG_FOLD_PAIRS if fold_pairs else MLA_FLAG_PER_TOKEN)
    flags = (MLA_FLAG_DEBUG_CHECKS if debug else 0) | (MLA_FLAG_KERNEL_TIMING if timing else 0) | walk
    return MlaOpts(mask=int(mask), window=int(window), scale=float(scale),
                   num_splits=int(num_splits), flags=flags)


def _buffer(shape, dtype, device, stream, returned=False):
    """A buffer of one call.  It comes from the memory of the stream that the call runs on: what
    another stream has given back may still be in use there.  One that is returned is not given to
    that stream again before the current stream is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def mla_decode_workspace_size(dims: MlaDims, opts: MlaOpts, batch: int, total_q: int) -> int:
    n = ctypes.c_size_t(0)
    rc = _lib.load().mla_decode_workspace_size(ctypes.byref(dims), ctypes.byref(opts), batch,
                                               total_q, ctypes.byref(n))
    if rc:
        raise MlaError("mla_decode_workspace_size", rc)
    return n.value


def _prepare(q, w_uk, w_uv, page_size, pool_bytes, row_bytes_fn, out, lse_out, workspace, opts,
             batch, stream):
    T, H, NR = q.shape
    Hk, L, N = w_uk.shape
    Hv, V, Lv = w_uv.shape
    if Hk != H or Hv != H or Lv != L:
        raise ValueError("q, w_uk and w_uv disagree on heads or latent width")
    R = NR - N
    row_bytes = row_bytes_fn(L, R)
    if pool_bytes % (page_size * row_bytes):
        raise ValueError("kv pool size is not a whole number of pages")
    dims = MlaDims(num_heads=H, qk_nope=N, qk_rope=R, kv_lora_rank=L, v_head=V,
                   page_size=page_size, num_pages=pool_bytes // (page_size * row_bytes))
    dev = q.device
    if out is None:
        out = _buffer((T, H, V), torch.bfloat16, dev, stream, returned=True)
    need = mla_decode_workspace_size(dims, opts, batch, T)
    if workspace is None:
        workspace = _buffer(max(need, 256), torch.uint8, dev, stream)
    return dims, out, workspace


def _stream(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def mla_decode_paged(q, input_row_offsets, kv_pool, block_table, cache_lens, w_uk, w_uv, *,
                     page_size: int, scale: Optional[float] = None, mask: int = MLA_MASK_CAUSAL,
                     window: int = 0, num_splits: int = 0, debug: bool = False, out=None,
                     lse_out=None, workspace=None, stream=None, timing: bool = False,
                     fold_pairs: Optional[bool] = None):
    """Dense bf16 decode.  Shapes as in include/mla_decode.h: q [T,H,N+R] bf16,
    input_row_offsets uint32/int32 [B+1], kv_pool bf16 (any shape, page-major rows of
    L+R), block_table int32 [B, stride], cache_lens uint32/int32 [B], w_uk [H,L,N],
    w_uv [H,V,L] bf16.  Returns (out [T,H,V] bf16, lse_out or None)."""
    dev = q.device
    B = input_row_offsets.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[2])
    opts = _opts(mask, window, scale, num_splits, debug, timing, fold_pairs)
    dims, out, workspace = _prepare(q, w_uk, w_uv, page_size,
                                    kv_pool.numel() * kv_pool.element_size(),
                                    lambda L, R: 2 * (L + R), out, lse_out, workspace, opts, B, stream)
    i32 = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
    rc = _lib.load().mla_decode_paged(
        ctypes.byref(dims), ctypes.byref(opts), _ptr(q, "q", (torch.bfloat16,), dev),
        _ptr(input_row_offsets, "input_row_offsets", i32, dev), B, q.shape[0],
        _ptr(kv_pool, "kv_pool", None, dev), _ptr(block_table, "block_table", (torch.int32,), dev),
        block_table.shape[1], _ptr(cache_lens, "cache_lens", i32, dev),
        _ptr(w_uk, "w_uk", (torch.bfloat16,), dev), _ptr(w_uv, "w_uv", (torch.bfloat16,), dev),
        _ptr(out, "out", (torch.bfloat16,), dev), _ptr(lse_out, "lse_out", (torch.float32,), dev),
        _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size(),
        _stream(stream, dev))
    if rc:
        raise MlaError("mla_decode_paged", rc)
    return out, lse_out


def mla_decode_paged_fp8(q, input_row_offsets, kv_pool_fp8, kv_scales, block_table, cache_lens,
                         w_uk_fp8, w_uk_scale, w_uv_fp8, w_uv_scale, *, page_size: int,
                         scale: Optional[float] = None, mask: int = MLA_MASK_CAUSAL,
                         window: int = 0, num_splits: int = 0, debug: bool = False, out=None,
                         lse_out=None, workspace=None, stream=None, q_scale=None,
                         timing: bool = False, fold_pairs: Optional[bool] = None):
    """FP8 latent cache: kv_pool_fp8 uint8 rows [L e4m3 | R bf16], kv_scales f32 [rows],
    e4m3 weights (uint8 or float8_e4m3fn) with fp32 128x128 block scales."""
    dev = q.device
    B = input_row_offsets.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[2])
    opts = _opts(mask, window, scale, num_splits, debug, timing, fold_pairs)
    dims, out, workspace = _prepare(q, w_uk_fp8, w_uv_fp8, page_size,
                                    kv_pool_fp8.numel() * kv_pool_fp8.element_size(),
                                    lambda L, R: L + 2 * R, out, lse_out, workspace, opts, B, stream)
    i32 = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
    f8 = (torch.uint8, torch.float8_e4m3fn)
    rc = _lib.load().mla_decode_paged_fp8(
        ctypes.byref(dims), ctypes.byref(opts), _ptr(q, "q", (torch.bfloat16,), dev),
        _ptr(input_row_offsets, "input_row_offsets", i32, dev), B, q.shape[0],
        _ptr(kv_pool_fp8, "kv_pool_fp8", None, dev), _ptr(kv_scales, "kv_scales", (torch.float32,), dev),
        _ptr(block_table, "block_table", (torch.int32,), dev), block_table.shape[1],
        _ptr(cache_lens, "cache_lens", i32, dev), _ptr(w_uk_fp8, "w_uk_fp8", f8, dev),
        _ptr(w_uk_scale, "w_uk_scale", (torch.float32,), dev), _ptr(w_uv_fp8, "w_uv_fp8", f8, dev),
        _ptr(w_uv_scale, "w_uv_scale", (torch.float32,), dev),
        _ptr(q_scale, "q_scale", (torch.float32,), dev),
        _ptr(out, "out", (torch.bfloat16,), dev), _ptr(lse_out, "lse_out", (torch.float32,), dev),
        _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size(),
        _stream(stream, dev))
    if rc:
        raise MlaError("mla_decode_paged_fp8", rc)
    return out, lse_out


_I32 = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
_BF16 = (torch.bfloat16,)


_status = {}


def _unread_status(device, stream):
    """The status word of a stream's calls that nobody reads it of: kernels only set bits in it."""
    key = (device.index, stream.cuda_stream)
    t = _status.get(key)
    if t is None:
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return torch.empty(256, dtype=torch.uint8, device=device)   # the graph's own memory, not kept
            t = _status[key] = torch.zeros(256, dtype=torch.uint8, device=device)
    return t


def _call(name, device, *args):
    """One library call with `device` current (the library launches on the current device)."""
    fn = getattr(_lib.load(), name)
    if device.index is None or torch.cuda.current_device() == device.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc:
        raise MlaError(name, rc)


def _tables(input_row_offsets, block_table, cache_lens, dev):
    B = input_row_offsets.numel() - 1
    if B < 1 or block_table.dim() != 2 or block_table.shape[0] < B or cache_lens.numel() < B:
        raise ValueError("input_row_offsets, block_table and cache_lens disagree on the number of requests")
    return (B, _ptr(input_row_offsets, "input_row_offsets", _I32, dev),
            _ptr(block_table, "block_table", (torch.int32,), dev), block_table.shape[1],
            _ptr(cache_lens, "cache_lens", _I32, dev))


def mla_cache_row_bytes(cache_format: int, kv_lora_rank: int, qk_rope: int) -> int:
    """Bytes of a cache row in a MLA_CACHE_ format."""
    L, R = int(kv_lora_rank), int(qk_rope)
    if cache_format == MLA_CACHE_BF16:
        return 2 * (L + R)
    if cache_format == MLA_CACHE_E4M3:
        return L + 2 * R
    if cache_format == MLA_CACHE_E2M1:
        return (L // 2 + L // 32 + 15) // 16 * 16 + 2 * R
    raise ValueError(f"unknown cache format {cache_format}")


def _pages(kv_pool, page_size, row_bytes):
    size = kv_pool.numel() * kv_pool.element_size()
    if page_size < 1 or size % (page_size * row_bytes):
        raise ValueError("kv pool size is not a whole number of pages")
    return size // (page_size * row_bytes)


def mla_cache_append(kv_new, input_row_offsets, kv_pool, block_table, cache_lens, freqs_cis,
                     kv_norm_gamma, *, page_size: int, epsilon: float,
                     cache_format: int = MLA_CACHE_BF16, kv_scales=None, q=None, q_out=None,
                     rows_out=None, debug: bool = False, workspace=None, stream=None):
    """New latent rows into the paged cache.  kv_new bf16 [T, L+R] (rows may be strided: a slice
    of a wider projection), normalised, turned and stored in `cache_format` at each token's
    position; kv_pool holds page-major rows of mla_cache_row_bytes() bytes, kv_scales f32 [rows]
    for MLA_CACHE_E4M3.  q bf16 [T,H,N+R] is turned into q_out (in place if q_out is None).
    rows_out bf16 [T, L+R] receives the values the written rows stand for.  freqs_cis bf16
    [max_seq_len, R], kv_norm_gamma bf16 [L].  Returns (kv_pool, q_out or None)."""
    dev = kv_new.device
    T = kv_new.shape[0]
    L, R = kv_norm_gamma.numel(), freqs_cis.shape[1]
    if kv_new.dim() != 2 or kv_new.shape[1] != L + R or (T > 0 and kv_new.stride(1) != 1):
        raise ValueError("kv_new must be [T, L+R] with unit stride along a row")
    if kv_new.dtype != torch.bfloat16 or not kv_new.is_cuda:
        raise TypeError("kv_new must be a bf16 CUDA tensor")
    new_stride = kv_new.stride(0) if T > 1 else -(-(L + R) // 8) * 8
    H, N = 1, 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] < R:
            raise ValueError("q must be [T, H, N+R]")
        H, N = q.shape[1], q.shape[2] - R
        q_out = q if q_out is None else q_out
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if rows_out is not None and tuple(rows_out.shape) != (T, L + R):
        raise ValueError("rows_out must be [T, L+R]")
    dims = MlaDims(num_heads=H, qk_nope=N, qk_rope=R, kv_lora_rank=L, v_head=1, page_size=page_size,
                   num_pages=_pages(kv_pool, page_size, mla_cache_row_bytes(cache_format, L, R)))
    if kv_scales is not None and kv_scales.numel() != dims.num_pages * page_size:
        raise ValueError("kv_scales must hold one value per cache row")
    B, offsets, table, table_stride, lens = _tables(input_row_offsets, block_table, cache_lens, dev)
    s = torch.cuda.current_stream(dev) if stream is None else stream
    if workspace is None:
        workspace = _buffer(256, torch.uint8, dev, stream) if debug else _unread_status(dev, s)
    _call("mla_cache_append", dev, ctypes.byref(dims), int(cache_format), kv_new.data_ptr(), new_stride, offsets,
          B, T, _ptr(q, "q", _BF16, dev), _ptr(q_out, "q_out", _BF16, dev), _ptr(kv_pool, "kv_pool", None, dev),
          _ptr(kv_scales, "kv_scales", (torch.float32,), dev), _ptr(rows_out, "rows_out", _BF16, dev), table,
          table_stride, lens, _ptr(freqs_cis, "freqs_cis", _BF16, dev), freqs_cis.shape[0],
          _ptr(kv_norm_gamma, "kv_norm_gamma", _BF16, dev), float(epsilon),
          MLA_FLAG_DEBUG_CHECKS if debug else 0, _ptr(workspace, "workspace", None, dev),
          workspace.numel() * workspace.element_size(), ctypes.c_void_p(s.cuda_stream))
    return kv_pool, q_out


def mla_decode_paged_fp4(q, input_row_offsets, kv_pool_fp4, block_table, cache_lens, w_uk, w_uv, *,
                         page_size: int, scale: Optional[float] = None, mask: int = MLA_MASK_CAUSAL,
                         window: int = 0, num_splits: int = 0, debug: bool = False, out=None,
                         lse_out=None, workspace=None, stream=None, timing: bool = False):
    """4-bit latent cache: kv_pool_fp4 uint8, page-major MLA_CACHE_E2M1 rows (e2m1 codes, e8m0
    scales of 32 values, bf16 rope).  Other arguments and results as mla_decode_paged."""
    dev = q.device
    T, H, NR = q.shape
    L, N = w_uk.shape[1:]
    V = w_uv.shape[1]
    if w_uk.shape[0] != H or tuple(w_uv.shape) != (H, V, L) or NR < N:
        raise ValueError("q, w_uk and w_uv disagree on heads or widths")
    B, offsets, table, table_stride, lens = _tables(input_row_offsets, block_table, cache_lens, dev)
    opts = _opts(mask, window, 1.0 / math.sqrt(NR) if scale is None else scale, num_splits, debug, timing)
    dims = MlaDims(num_heads=H, qk_nope=N, qk_rope=NR - N, kv_lora_rank=L, v_head=V, page_size=page_size,
                   num_pages=_pages(kv_pool_fp4, page_size, mla_cache_row_bytes(MLA_CACHE_E2M1, L, NR - N)))
    if out is None:
        out = _buffer((T, H, V), torch.bfloat16, dev, stream, returned=True)
    elif tuple(out.shape) != (T, H, V):
        raise ValueError("out must be [T, H, V]")
    if lse_out is not None and lse_out.numel() != T * H:
        raise ValueError("lse_out must be [T, H]")
    if T == 0:
        return out, lse_out
    if workspace is None:
        n = ctypes.c_size_t(0)
        _call("mla_decode_workspace_size", dev, ctypes.byref(dims), ctypes.byref(opts), B, T, ctypes.byref(n))
        workspace = _buffer(max(n.value, 256), torch.uint8, dev, stream)
    _call("mla_decode_paged_fp4", dev, ctypes.byref(dims), ctypes.byref(opts), _ptr(q, "q", _BF16, dev), offsets, B,
          T, _ptr(kv_pool_fp4, "kv_pool_fp4", None, dev), table, table_stride, lens, _ptr(w_uk, "w_uk", _BF16, dev),
          _ptr(w_uv, "w_uv", _BF16, dev), _ptr(out, "out", _BF16, dev),
          _ptr(lse_out, "lse_out", (torch.float32,), dev), _ptr(workspace, "workspace", None, dev),
          workspace.numel() * workspace.element_size(), _stream(stream, dev))
    return out, lse_out


def mla_prefill_workspace_size(dims: MlaDims, opts: MlaOpts, cache_format: int, batch: int,
                               total_q: int, total_keys: int) -> int:
    n = ctypes.c_size_t(0)
    rc = _lib.load().mla_prefill_workspace_size(ctypes.byref(dims), ctypes.byref(opts), int(cache_format), batch,
                                                total_q, int(total_keys), ctypes.byref(n))
    if rc:
        raise MlaError("mla_prefill_workspace_size", rc)
    return n.value


def _prefill(name, cache_format, q, input_row_offsets, cache, block_table, cache_lens, w_uk, w_uv, weights, *,
             page_size, total_keys, scale, mask, window, num_splits, debug, out, lse_out, workspace, stream):
    dev = q.device
    T, H, NR = q.shape
    L, N = w_uk.shape[1:]
    V = w_uv.shape[1]
    if w_uk.shape[0] != H or tuple(w_uv.shape) != (H, V, L) or NR < N:
        raise ValueError("q, w_uk and w_uv disagree on heads or widths")
    B, offsets, table, table_stride, lens = _tables(input_row_offsets, block_table, cache_lens, dev)
    opts = _opts(mask, window, 1.0 / math.sqrt(NR) if scale is None else scale, num_splits, debug)
    dims = MlaDims(num_heads=H, qk_nope=N, qk_rope=NR - N, kv_lora_rank=L, v_head=V, page_size=page_size,
                   num_pages=_pages(cache[0], page_size, mla_cache_row_bytes(cache_format, L, NR - N)))
    if len(cache) > 1 and cache[1].numel() != dims.num_pages * page_size:
        raise ValueError("kv_scales must hold one value per cache row")
    if out is None:
        out = _buffer((T, H, V), torch.bfloat16, dev, stream, returned=True)
    elif tuple(out.shape) != (T, H, V):
        raise ValueError("out must be [T, H, V]")
    if lse_out is not None and lse_out.numel() != T * H:
        raise ValueError("lse_out must be [T, H]")
    if T == 0:
        return out, lse_out
    if workspace is None:
        n = ctypes.c_size_t(0)
        _call("mla_prefill_workspace_size", dev, ctypes.byref(dims), ctypes.byref(opts), cache_format, B, T,
              int(total_keys), ctypes.byref(n))
        workspace = _buffer(n.value, torch.uint8, dev, stream)
    pools = [_ptr(cache[0], "kv_pool", None, dev)]
    if len(cache) > 1:
        pools.append(_ptr(cache[1], "kv_scales", (torch.float32,), dev))
    _call(name, dev, ctypes.byref(dims), ctypes.byref(opts), _ptr(q, "q", _BF16, dev), offsets, B, T, *pools, table,
          table_stride, lens, int(total_keys), *weights, _ptr(out, "out", _BF16, dev),
          _ptr(lse_out, "lse_out", (torch.float32,), dev), _ptr(workspace, "workspace", None, dev),
          workspace.numel() * workspace.element_size(), _stream(stream, dev))
    return out, lse_out


def mla_prefill_paged(q, input_row_offsets, kv_pool, block_table, cache_lens, w_uk, w_uv, *, page_size: int,
                      total_keys: int, scale: Optional[float] = None, mask: int = MLA_MASK_CAUSAL, window: int = 0,
                      num_splits: int = 0, debug: bool = False, out=None, lse_out=None, workspace=None,
                      stream=None):
    """Prefill over a bf16 latent cache, in the expanded form: arguments and results of
    mla_decode_paged, for many query tokens per request.  total_keys (host) bounds the sum of
    the requests' cached tokens and sizes the workspace."""
    dev = q.device
    return _prefill("mla_prefill_paged", MLA_CACHE_BF16, q, input_row_offsets, (kv_pool,), block_table, cache_lens,
                    w_uk, w_uv, (_ptr(w_uk, "w_uk", _BF16, dev), _ptr(w_uv, "w_uv", _BF16, dev)),
                    page_size=page_size, total_keys=total_keys, scale=scale, mask=mask, window=window,
                    num_splits=num_splits, debug=debug, out=out, lse_out=lse_out, workspace=workspace, stream=stream)


def mla_prefill_paged_fp8(q, input_row_offsets, kv_pool_fp8, kv_scales, block_table, cache_lens, w_uk_fp8, w_uk_scale,
                          w_uv_fp8, w_uv_scale, *, page_size: int, total_keys: int, scale: Optional[float] = None,
                          mask: int = MLA_MASK_CAUSAL, window: int = 0, num_splits: int = 0, debug: bool = False,
                          out=None, lse_out=None, workspace=None, stream=None):
    """mla_prefill_paged over the e4m3 cache and weights of mla_decode_paged_fp8."""
    dev = q.device
    f8, f32 = (torch.uint8, torch.float8_e4m3fn), (torch.float32,)
    for w, s, name in ((w_uk_fp8, w_uk_scale, "w_uk_scale"), (w_uv_fp8, w_uv_scale, "w_uv_scale")):
        if s.numel() != w.shape[0] * (-(-w.shape[1] // 128)) * (-(-w.shape[2] // 128)):
            raise ValueError(f"{name} must hold one value per 128 x 128 block")
    weights = (_ptr(w_uk_fp8, "w_uk_fp8", f8, dev), _ptr(w_uk_scale, "w_uk_scale", f32, dev),
               _ptr(w_uv_fp8, "w_uv_fp8", f8, dev), _ptr(w_uv_scale, "w_uv_scale", f32, dev))
    return _prefill("mla_prefill_paged_fp8", MLA_CACHE_E4M3, q, input_row_offsets, (kv_pool_fp8, kv_scales),
                    block_table, cache_lens, w_uk_fp8, w_uv_fp8, weights, page_size=page_size, total_keys=total_keys,
                    scale=scale, mask=mask, window=window, num_splits=num_splits, debug=debug, out=out,
                    lse_out=lse_out, workspace=workspace, stream=stream)


def mla_prefill_paged_fp4(q, input_row_offsets, kv_pool_fp4, block_table, cache_lens, w_uk, w_uv, *, page_size: int,
                          total_keys: int, scale: Optional[float] = None, mask: int = MLA_MASK_CAUSAL,
                          window: int = 0, num_splits: int = 0, debug: bool = False, out=None, lse_out=None,
                          workspace=None, stream=None):
    """mla_prefill_paged over the 4-bit cache of mla_decode_paged_fp4."""
    dev = q.device
    return _prefill("mla_prefill_paged_fp4", MLA_CACHE_E2M1, q, input_row_offsets, (kv_pool_fp4,), block_table,
                    cache_lens, w_uk, w_uv, (_ptr(w_uk, "w_uk", _BF16, dev), _ptr(w_uv, "w_uv", _BF16, dev)),
                    page_size=page_size, total_keys=total_keys, scale=scale, mask=mask, window=window,
                    num_splits=num_splits, debug=debug, out=out, lse_out=lse_out, workspace=workspace, stream=stream)


def mla_decode_sparse(q, input_row_offsets, kv_pool, d_indices, topk_lengths, w_uk, w_uv, *,
                      page_size: int, scale: Optional[float] = None, num_splits: int = 0,
                      debug: bool = False, out=None, lse_out=None, workspace=None, stream=None,
                      timing: bool = False, fold_pairs: Optional[bool] = None):
    """Sparse top-k decode over physical rows d_indices int32 [B, stride] (-1 = skip);
    topk_lengths int32 [B] or None."""
    dev = q.device
    B = input_row_offsets.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[2])
    opts = _opts(MLA_MASK_NULL, 0, scale, num_splits, debug, timing, fold_pairs)
    dims, out, workspace = _prepare(q, w_uk, w_uv, page_size,
                                    kv_pool.numel() * kv_pool.element_size(),
                                    lambda L, R: 2 * (L + R), out, lse_out, workspace, opts, B, stream)
    i32 = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
    rc = _lib.load().mla_decode_sparse(
        ctypes.byref(dims), ctypes.byref(opts), _ptr(q, "q", (torch.bfloat16,), dev),
        _ptr(input_row_offsets, "input_row_offsets", i32, dev), B, q.shape[0],
        _ptr(kv_pool, "kv_pool", None, dev), _ptr(d_indices, "d_indices", (torch.int32,), dev),
        d_indices.shape[1], _ptr(topk_lengths, "topk_lengths", (torch.int32,), dev),
        _ptr(w_uk, "w_uk", (torch.bfloat16,), dev), _ptr(w_uv, "w_uv", (torch.bfloat16,), dev),
        _ptr(out, "out", (torch.bfloat16,), dev), _ptr(lse_out, "lse_out", (torch.float32,), dev),
        _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size(),
        _stream(stream, dev))
    if rc:
        raise MlaError("mla_decode_sparse", rc)
    return out, lse_out


def mla_branch_prologue(q, input_row_offsets, kv_pool, block_table, cache_lens, freqs_cis,
                        kv_norm_gamma, *, page_size: int, kv_lora_rank: int, epsilon: float,
                        debug: bool = False, workspace=None, stream=None):
    """In place: RoPE on q's rope part and, per query token, RMSNorm + RoPE of the cache
    row at its position.  q bf16 [T,H,N+R]; kv_pool bf16 rows of L+R (L = kv_lora_rank);
    freqs_cis bf16 [max_seq_len, R]; kv_norm_gamma bf16 [L].  Returns (q, kv_pool)."""
    dev = q.device
    T, H, NR = q.shape
    B = input_row_offsets.numel() - 1
    L = int(kv_lora_rank)
    R = freqs_cis.shape[1]
    row_bytes = 2 * (L + R)
    pool_bytes = kv_pool.numel() * kv_pool.element_size()
    if pool_bytes % (page_size * row_bytes):
        raise ValueError("kv pool size is not a whole number of pages")
    dims = MlaDims(num_heads=H, qk_nope=NR - R, qk_rope=R, kv_lora_rank=L, v_head=1,
                   page_size=page_size, num_pages=pool_bytes // (page_size * row_bytes))
    if workspace is None:
        workspace = _buffer(256, torch.uint8, dev, stream)
    i32 = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
    rc = _lib.load().mla_branch_prologue(
        ctypes.byref(dims), _ptr(q, "q", (torch.bfloat16,), dev),
        _ptr(input_row_offsets, "input_row_offsets", i32, dev), B, T,
        _ptr(kv_pool, "kv_pool", None, dev), _ptr(block_table, "block_table", (torch.int32,), dev),
        block_table.shape[1], _ptr(cache_lens, "cache_lens", i32, dev),
        _ptr(freqs_cis, "freqs_cis", (torch.bfloat16,), dev), freqs_cis.shape[0],
        _ptr(kv_norm_gamma, "kv_norm_gamma", (torch.bfloat16,), dev), float(epsilon),
        MLA_FLAG_DEBUG_CHECKS if debug else 0,
        _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size(),
        _stream(stream, dev))
    if rc:
        raise MlaError("mla_branch_prologue", rc)
    return q, kv_pool


def mla_indexer_fp8(q, q_s, input_row_offsets, k_cache, k_scales, block_table, cache_lens, *,
                    page_size: int, top_k: int, mask: int = MLA_MASK_CAUSAL, window: int = 0,
                    with_scores: bool = False, debug: bool = False, out=None, workspace=None,
                    stream=None):
    """Top-k physical cache rows per query token.  q e4m3 codes [T,H,D] (uint8 or
    float8_e4m3fn), q_s f32 [T,H], k_cache e4m3 codes (page-major rows of D), k_scales f32
    [rows].  Returns (indices int32 [T, top_k], scores f64 [T, top_k] or None)."""
    dev = q.device
    T, H, D = q.shape
    B = input_row_offsets.numel() - 1
    rows = k_cache.numel() // D
    if rows % page_size:
        raise ValueError("k_cache is not a whole number of pages")
    lib = _lib.load()
    need = ctypes.c_size_t(0)
    rc = lib.mla_indexer_workspace_size(T, block_table.shape[1], page_size, int(mask), int(window),
                                        ctypes.byref(need))
    if rc:
        raise MlaError("mla_indexer_workspace_size", rc)
    if workspace is None:
        workspace = _buffer(need.value, torch.uint8, dev, stream)
    if out is None:
        out = _buffer((T, top_k), torch.int32, dev, stream, returned=True)
    scores = _buffer((T, top_k), torch.float64, dev, stream, returned=True) if with_scores else None
    i32 = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
    f8 = (torch.uint8, torch.float8_e4m3fn)
    rc = lib.mla_indexer_fp8(
        H, D, page_size, rows // page_size, _ptr(q, "q", f8, dev), _ptr(q_s, "q_s", (torch.float32,), dev),
        _ptr(input_row_offsets, "input_row_offsets", i32, dev), B, T,
        _ptr(k_cache, "k_cache", f8, dev), _ptr(k_scales, "k_scales", (torch.float32,), dev),
        _ptr(block_table, "block_table", (torch.int32,), dev), block_table.shape[1],
        _ptr(cache_lens, "cache_lens", i32, dev), int(mask), int(window), int(top_k),
        _ptr(out, "out", (torch.int32,), dev), _ptr(scores, "scores", (torch.float64,), dev),
        MLA_FLAG_DEBUG_CHECKS if debug else 0,
        _ptr(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size(),
        _stream(stream, dev))
    if rc:
        raise MlaError("mla_indexer_fp8", rc)
    return out, scores
