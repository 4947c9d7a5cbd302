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
  mla_cache_read        cache rows of any format back as bf16 values
  mla_rmsnorm_quant     residual addition, RMSNorm and 8-bit codes (e4m3, int8) of activations
  mla_linear_fp8        projections over e4m3 codes with scales per token and channel (also _int8)
  mla_indexer_append    the indexer's keys (LayerNorm, RoPE, e4m3) into its paged cache, its queries as codes
  mla_indexer_fp8       top-k cache rows per query token by FP8 index scores (sparse input)
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch

from . import _lib
from ._lib import (MLA_FLAG_DEBUG_CHECKS, MLA_FLAG_KERNEL_TIMING, MLA_FLAG_FOLD_PAIRS, MLA_FLAG_PER_TOKEN,
                   MLA_CACHE_BF16, MLA_CACHE_E2M1, MLA_CACHE_E4M3, MLA_CODES_BF16, MLA_CODES_E4M3, MLA_CODES_INT8,
                   MLA_MASK_CAUSAL, MLA_MASK_NULL,
                   MLA_MASK_SLIDING_WINDOW_CAUSAL, MlaDims, MlaError, MlaOpts, kernel_times)

__all__ = ["mla_decode_paged", "mla_decode_paged_fp8", "mla_decode_paged_fp4", "mla_decode_sparse",
           "mla_branch_prologue", "mla_cache_append", "mla_cache_row_bytes", "mla_indexer_fp8",
           "mla_prefill_paged", "mla_prefill_paged_fp8", "mla_prefill_paged_fp4", "mla_prefill_workspace_size",
           "mla_cache_read", "mla_rmsnorm_quant", "mla_linear_fp8", "mla_linear_int8", "mla_indexer_append",
           "MLA_CACHE_BF16", "MLA_CACHE_E4M3", "MLA_CACHE_E2M1", "MLA_CODES_BF16", "MLA_CODES_E4M3", "MLA_CODES_INT8",
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
_INT32 = (torch.int32,)
_INT8 = (torch.int8, torch.uint8)
_F8 = (torch.float8_e4m3fn, torch.uint8)
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)


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


def _handle(stream, device):
    """The cudaStream_t that a call runs on, without a Stream object for the current one (3 us of a call)."""
    if device.index is None:
        raise ValueError(f"tensors must be CUDA tensors, not on {device}")
    # looked up here, not at import: a torch without CUDA has neither name, and the host functions need none
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _status_word(workspace, debug, device, stream, handle):
    """Pointer and size of a call's status word: the caller's workspace, one of its own where it is read."""
    if workspace is None:
        if debug:
            workspace = _buffer(256, torch.uint8, device, stream)
        else:
            workspace = _status.get((device.index, handle))
            if workspace is not None:
                return workspace.data_ptr(), 256, workspace
            workspace = _unread_status(device, torch.cuda.current_stream(device) if stream is None else stream)
    return _ptr(workspace, "workspace", None, device), workspace.numel() * workspace.element_size(), workspace


def _at(t, name, dtypes, index):
    """_ptr of a tensor that is right, by its cheapest attributes; what is not goes to _ptr, which says why."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype in dtypes and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, name, dtypes, torch.device("cuda", index))


def _bytes_at(t, name, index):
    """_at of a tensor of any type."""
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, name, None, torch.device("cuda", index))


_fns = {}


def _call(name, device, *args):
    """One library call with `device` current (the library launches on the current device)."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_lib.load(), name)
    if device.index is None or torch._C._cuda_getDevice() == device.index:
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
    i = dev.index
    if i is None:
        raise ValueError(f"tensors must be CUDA tensors, not on {dev}")
    return (B, _at(input_row_offsets, "input_row_offsets", _I32, i), _at(block_table, "block_table", _INT32, i),
            block_table.shape[1], _at(cache_lens, "cache_lens", _I32, i))


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


def _row_strided(t, name, width, index):
    """Pointer and row stride of a bf16 CUDA tensor whose rows may lie apart (a slice of a wider one)."""
    if t.dtype != torch.bfloat16 or t.get_device() != index:
        raise TypeError(f"{name} must be a bf16 tensor on cuda:{index}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name} must be [rows, {width}]")
    by_row, along = t.stride()
    if along != 1 and shape[0] > 0:
        raise ValueError(f"{name} must have unit stride along a row")
    return t.data_ptr(), by_row if shape[0] > 1 else -(-width // 8) * 8


def _out(t, name, dtypes, shape, index):
    """Pointer of a given output of that shape."""
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return _at(t, name, dtypes, index)


def _sized(t, name, n):
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must hold {n} values")


@functools.lru_cache(maxsize=64)
def _cache_dims(L, R, page_size, num_pages):
    return MlaDims(num_heads=1, qk_nope=0, qk_rope=R, kv_lora_rank=L, v_head=1, page_size=page_size, num_pages=num_pages)


def mla_cache_read(input_row_offsets, kv_pool, block_table, cache_lens, *, kv_lora_rank: int, qk_rope: int,
                   page_size: int, total_rows: Optional[int] = None, cache_format: int = MLA_CACHE_BF16, kv_scales=None,
                   out=None, debug: bool = False, workspace=None, stream=None):
    """Cache rows back as bf16 values: the last input_row_offsets[b+1] - input_row_offsets[b] of request b's
    cache_lens[b] tokens.  total_rows (host) is input_row_offsets' last value; it may be left out where `out`
    bf16 [total_rows, L+R] is given.  Returns out."""
    dev, L, R, page_size = kv_pool.device, int(kv_lora_rank), int(qk_rope), int(page_size)
    i, handle = dev.index, _handle(stream, dev)
    num_pages = _pages(kv_pool, page_size, mla_cache_row_bytes(cache_format, L, R))
    _sized(kv_scales, "kv_scales", num_pages * page_size)
    B, offsets, table, table_stride, lens = _tables(input_row_offsets, block_table, cache_lens, dev)
    if out is None:
        if total_rows is None:
            raise ValueError("total_rows or out must be given")
        out = _buffer((total_rows, L + R), torch.bfloat16, dev, stream, returned=True)
        p_out = out.data_ptr()
    else:
        total_rows = out.shape[0] if total_rows is None else total_rows
        p_out = _out(out, "out", _BF16, (total_rows, L + R), i)
    status, status_bytes, workspace = _status_word(workspace, debug, dev, stream, handle)
    _call("mla_cache_read", dev, ctypes.byref(_cache_dims(L, R, page_size, num_pages)), int(cache_format), offsets, B,
          total_rows, _bytes_at(kv_pool, "kv_pool", i), _at(kv_scales, "kv_scales", _F32, i), table, table_stride, lens,
          p_out, MLA_FLAG_DEBUG_CHECKS if debug else 0, status, status_bytes, handle)
    return out


_CODES = {MLA_CODES_BF16: (), MLA_CODES_E4M3: (torch.float8_e4m3fn, torch.uint8),
          MLA_CODES_INT8: (torch.int8, torch.uint8)}


def mla_rmsnorm_quant(x, gamma=None, *, epsilon: float = 1e-6, code_format: int = MLA_CODES_E4M3, residual=None,
                      residual_out=None, y_out=None, codes_out=None, scales_out=None, stream=None):
    """Rows x bf16 [T, D] (rows may be strided) plus residual bf16 [T, D], normalised by gamma bf16 [D] (as they
    are without it), as e4m3 or int8 codes with one fp32 scale a row.  The sum goes to residual_out (in place if
    it is None); y_out bf16 [T, D] receives the normalised rows.  Returns (codes [T, D], scales [T],
    residual_out or None); for MLA_CODES_BF16 (y_out, None, residual_out or None)."""
    dev, shape = x.device, tuple(x.shape)
    i, handle = dev.index, _handle(stream, dev)
    if len(shape) != 2:
        raise ValueError("x must be [T, D]")
    if code_format not in _CODES:
        raise ValueError(f"unknown code format {code_format}")
    T, D = shape
    px, stride = _row_strided(x, "x", D, i)
    p_res = p_res_out = p_gamma = p_y = p_codes = p_scales = None
    if residual is not None:
        residual_out = residual if residual_out is None else residual_out
        p_res = _out(residual, "residual", _BF16, shape, i)
        p_res_out = p_res if residual_out is residual else _out(residual_out, "residual_out", _BF16, shape, i)
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    if gamma is not None:
        _sized(gamma, "gamma", D)
        p_gamma = _at(gamma, "gamma", _BF16, i)
    coded = code_format != MLA_CODES_BF16
    if not coded:
        if codes_out is not None or scales_out is not None:
            raise ValueError("MLA_CODES_BF16 writes no codes")
        if y_out is None:
            y_out = _buffer(shape, torch.bfloat16, dev, stream, returned=True)
    else:
        if codes_out is None:
            codes_out = _buffer(shape, _CODES[code_format][0], dev, stream, returned=True)
            p_codes = codes_out.data_ptr()
        else:
            p_codes = _out(codes_out, "codes_out", _CODES[code_format], shape, i)
        if scales_out is None:
            scales_out = _buffer(T, torch.float32, dev, stream, returned=True)
            p_scales = scales_out.data_ptr()
        else:
            _sized(scales_out, "scales_out", T)
            p_scales = _at(scales_out, "scales_out", _F32, i)
    if y_out is not None:
        p_y = _out(y_out, "y_out", _BF16, shape, i)
    _call("mla_rmsnorm_quant", dev, code_format, T, D, px, stride, p_res, p_res_out, p_gamma, epsilon, p_y, p_codes,
          p_scales, handle)
    return (codes_out, scales_out, residual_out) if coded else (y_out, None, residual_out)


def _linear(name, dtypes, x_codes, x_scales, w_codes, w_scales, out, debug, workspace, stream):
    dev, x_shape, w_shape = x_codes.device, x_codes.shape, w_codes.shape
    i, handle = dev.index, _handle(stream, dev)
    if len(x_shape) != 2 or len(w_shape) != 2 or x_shape[1] != w_shape[1]:
        raise ValueError("x_codes must be [T, K] and w_codes [N, K]")
    T, K = x_shape
    N = w_shape[0]
    _sized(x_scales, "x_scales", T)
    _sized(w_scales, "w_scales", N)
    if out is None:
        out = _buffer((T, N), torch.bfloat16, dev, stream, returned=True)
        p_out, out_stride = out.data_ptr(), N
    else:
        if out.shape[0] != T:
            raise ValueError(f"out must be [{T}, {N}]")
        p_out, out_stride = _row_strided(out, "out", N, i)
    status, status_bytes, workspace = _status_word(workspace, debug, dev, stream, handle)
    _call(name, dev, T, N, K, _at(x_codes, "x_codes", dtypes, i), _at(x_scales, "x_scales", _F32, i),
          _at(w_codes, "w_codes", dtypes, i), _at(w_scales, "w_scales", _F32, i), p_out, out_stride,
          MLA_FLAG_DEBUG_CHECKS if debug else 0, status, status_bytes, handle)
    return out


def mla_linear_fp8(x_codes, x_scales, w_codes, w_scales, *, out=None, debug: bool = False, workspace=None, stream=None):
    """Projection over e4m3 codes: x_codes [T, K], w_codes [N, K] (float8_e4m3fn or uint8), x_scales f32 [T],
    w_scales f32 [N].  Returns out bf16 [T, N] (rows may be strided if given)."""
    return _linear("mla_linear_fp8", _F8, x_codes, x_scales, w_codes, w_scales, out, debug, workspace, stream)


def mla_linear_int8(x_codes, x_scales, w_codes, w_scales, *, out=None, debug: bool = False, workspace=None, stream=None):
    """mla_linear_fp8 over int8 codes (int8, or uint8 that holds them)."""
    return _linear("mla_linear_int8", _INT8, x_codes, x_scales, w_codes, w_scales, out, debug, workspace, stream)


def mla_indexer_append(k_new, input_row_offsets, k_cache, k_scales, block_table, cache_lens, *, page_size: int,
                       freqs_cis=None, k_norm_gamma=None, k_norm_beta=None, epsilon: float = 1e-6, q=None,
                       q_weight=None, q_codes=None, q_scales=None, debug: bool = False, workspace=None, stream=None):
    """The inputs of mla_indexer_fp8: keys k_new bf16 [T, D] (rows may be strided) through LayerNorm
    (k_norm_gamma, k_norm_beta bf16 [D]) and RoPE of their last R values (freqs_cis bf16 [max_seq_len, R]) into the
    e4m3 cache k_cache (page-major rows of D) with k_scales f32 [rows]; queries q bf16 [T, H, D] turned and coded,
    their scales times q_weight f32 [T, H].  Returns (q_codes e4m3 [T, H, D], q_scales f32 [T, H]) or (None, None)."""
    dev, shape = k_new.device, k_new.shape
    i, handle = dev.index, _handle(stream, dev)
    if len(shape) != 2:
        raise ValueError("k_new must be [T, D]")
    T, D = shape
    pk, stride = _row_strided(k_new, "k_new", D, i)
    R, max_len = (freqs_cis.shape[1], freqs_cis.shape[0]) if freqs_cis is not None else (0, 0)
    num_pages = _pages(k_cache, page_size, D)
    _sized(k_scales, "k_scales", num_pages * page_size)
    _sized(k_norm_gamma, "k_norm_gamma", D)
    _sized(k_norm_beta, "k_norm_beta", D)
    H = 0
    if q is not None:
        if len(q.shape) != 3 or q.shape[0] != T or q.shape[2] != D:
            raise ValueError("q must be [T, H, D]")
        H = q.shape[1]
        if q_codes is None:
            q_codes = _buffer((T, H, D), torch.float8_e4m3fn, dev, stream, returned=True)
        if q_scales is None:
            q_scales = _buffer((T, H), torch.float32, dev, stream, returned=True)
        _sized(q_codes, "q_codes", T * H * D)
        _sized(q_scales, "q_scales", T * H)
        _sized(q_weight, "q_weight", T * H)
    elif q_weight is not None or q_codes is not None or q_scales is not None:
        raise ValueError("q_weight, q_codes or q_scales without q")
    B, offsets, table, table_stride, lens = _tables(input_row_offsets, block_table, cache_lens, dev)
    status, status_bytes, workspace = _status_word(workspace, debug, dev, stream, handle)
    _call("mla_indexer_append", dev, H, D, R, page_size, num_pages, pk, stride, offsets, B, T, _at(q, "q", _BF16, i),
          _at(q_weight, "q_weight", _F32, i), _at(q_codes, "q_codes", _F8, i), _at(q_scales, "q_scales", _F32, i),
          _at(k_cache, "k_cache", _F8, i), _at(k_scales, "k_scales", _F32, i), table, table_stride, lens,
          _at(freqs_cis, "freqs_cis", _BF16, i), max_len, _at(k_norm_gamma, "k_norm_gamma", _BF16, i),
          _at(k_norm_beta, "k_norm_beta", _BF16, i), epsilon, MLA_FLAG_DEBUG_CHECKS if debug else 0, status, status_bytes,
          handle)
    return q_codes, q_scales


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
