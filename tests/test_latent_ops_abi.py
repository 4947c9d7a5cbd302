"""CPU-side checks of the append, 4-bit decode and prefill entry points: what they refuse
before anything reaches a GPU, the workspace sizes, and the cache formats' reference."""
import ctypes

import numpy as np
import pytest
import torch

import mla_decode_attention_06_gb300 as M
import latent_ref as R

FAKE = 0x10000   # aligned, never dereferenced: every case below fails validation first
INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from mla_decode_attention_06_gb300 import _lib, build
    build.build()
    return _lib.load()


def _dims(**kw):
    d = dict(num_heads=128, qk_nope=128, qk_rope=64, kv_lora_rank=512, v_head=128, page_size=64, num_pages=100)
    d.update(kw)
    return M.MlaDims(**d)


def _opts(**kw):
    o = dict(mask=1, window=0, scale=0.07, num_splits=4, flags=0)
    o.update(kw)
    return M.MlaOpts(**o)


def _append(lib, dims=None, fmt=0, new=FAKE, stride=576, off=FAKE, B=2, T=2, q=FAKE, q_out=FAKE, pool=FAKE, scales=None,
            rows=None, table=FAKE, bt_stride=4, lens=FAKE, freqs=FAKE, max_seq=64, gamma=FAKE, eps=1e-6, flags=0,
            ws=FAKE, ws_bytes=1 << 20):
    return lib.mla_cache_append(ctypes.byref(dims or _dims()), fmt, new, stride, off, B, T, q, q_out, pool, scales,
                                rows, table, bt_stride, lens, freqs, max_seq, gamma, eps, flags, ws, ws_bytes, None)


def test_append_refuses_invalid_arguments(lib):
    for kw in (dict(new=None), dict(off=None), dict(pool=None), dict(table=None), dict(lens=None), dict(freqs=None),
               dict(gamma=None), dict(ws=None), dict(new=FAKE + 8), dict(q=FAKE + 8), dict(q_out=FAKE + 8),
               dict(pool=FAKE + 8), dict(rows=FAKE + 8), dict(freqs=FAKE + 8), dict(gamma=FAKE + 8),
               dict(fmt=-1), dict(fmt=3), dict(stride=568), dict(stride=580), dict(stride=0), dict(B=0), dict(T=-1),
               dict(bt_stride=0), dict(max_seq=0), dict(eps=-1.0), dict(eps=float("nan")), dict(flags=2), dict(flags=16),
               dict(q=None), dict(q_out=None),                 # queries come in and go out together
               dict(fmt=1), dict(fmt=0, scales=FAKE), dict(fmt=2, scales=FAKE),   # row scales for e4m3, and only there
               dict(dims=_dims(num_heads=0)), dict(dims=_dims(page_size=0)), dict(dims=_dims(num_pages=0)),
               dict(dims=_dims(kv_lora_rank=0)), dict(dims=_dims(qk_rope=0))):
        assert _append(lib, **kw) == INVALID, kw
    assert lib.mla_cache_append(None, 0, FAKE, 576, FAKE, 2, 2, None, None, FAKE, None, None, FAKE, 4, FAKE, FAKE, 64,
                                FAKE, 1e-6, 0, FAKE, 1 << 20, None) == INVALID


def test_append_reports_unsupported_shapes(lib):
    for kw in (dict(kv_lora_rank=520), dict(kv_lora_rank=544), dict(kv_lora_rank=48), dict(qk_rope=60),
               dict(qk_rope=136), dict(qk_nope=100), dict(page_size=1 << 20, num_pages=1 << 12)):
        assert _append(lib, dims=_dims(**kw), stride=1024) == UNSUPPORTED, kw
    assert _append(lib, dims=_dims(num_heads=1 << 24)) == UNSUPPORTED     # a token's queries pass 32 bits
    assert _append(lib, T=1 << 30, q_out=FAKE + 16) == UNSUPPORTED        # more blocks than a grid has
    assert _append(lib, T=1 << 30, ws_bytes=0, q=None, q_out=None) == TOO_SMALL
    # without queries the head count and qk_nope are not looked at; the workspace is
    assert _append(lib, dims=_dims(num_heads=0, qk_nope=-1), q=None, q_out=None, ws_bytes=0) == TOO_SMALL
    assert _append(lib, ws=FAKE + 8) == TOO_SMALL


def _fp4(lib, dims=None, opts=None, q=FAKE, pool=FAKE, table=FAKE, lens=FAKE, w=FAKE, out=FAKE, bt_stride=4,
         ws_bytes=1 << 40):
    return lib.mla_decode_paged_fp4(ctypes.byref(dims or _dims()), ctypes.byref(opts or _opts()), q, FAKE, 2, 2, pool,
                                    table, bt_stride, lens, w, w, out, None, FAKE, ws_bytes, None)


def test_fp4_decode_refuses_what_the_decode_refuses(lib):
    for kw in (dict(q=None), dict(q=FAKE + 2), dict(pool=None), dict(pool=FAKE + 8), dict(table=None), dict(lens=None),
               dict(w=None), dict(w=FAKE + 8), dict(out=None), dict(bt_stride=0), dict(opts=_opts(mask=7)),
               dict(opts=_opts(mask=2, window=0)), dict(opts=_opts(scale=float("nan"))), dict(opts=_opts(num_splits=-1)),
               dict(opts=_opts(flags=16)), dict(dims=_dims(num_heads=0))):
        assert _fp4(lib, **kw) == INVALID, kw
    for kw in (dict(num_heads=129), dict(kv_lora_rank=256), dict(page_size=48), dict(page_size=4), dict(qk_nope=100),
               dict(v_head=100)):
        assert _fp4(lib, dims=_dims(**kw)) == UNSUPPORTED, kw
    assert _fp4(lib, ws_bytes=1024) == TOO_SMALL


def _prefill(lib, fmt, dims=None, opts=None, q=FAKE, off=FAKE, B=2, T=2, pool=FAKE, scales=FAKE, table=FAKE, bt_stride=4,
             lens=FAKE, keys=1000, w=FAKE, w_scale=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    d, o = ctypes.byref(dims or _dims()), ctypes.byref(opts or _opts())
    if fmt == M.MLA_CACHE_E4M3:
        return lib.mla_prefill_paged_fp8(d, o, q, off, B, T, pool, scales, table, bt_stride, lens, keys, w, w_scale, w,
                                         w_scale, out, None, ws, ws_bytes, None)
    fn = lib.mla_prefill_paged if fmt == M.MLA_CACHE_BF16 else lib.mla_prefill_paged_fp4
    return fn(d, o, q, off, B, T, pool, table, bt_stride, lens, keys, w, w, out, None, ws, ws_bytes, None)


@pytest.mark.parametrize("fmt", [M.MLA_CACHE_BF16, M.MLA_CACHE_E4M3, M.MLA_CACHE_E2M1])
def test_prefill_refusals(lib, fmt):
    for kw in (dict(q=None), dict(off=None), dict(pool=None), dict(table=None), dict(lens=None), dict(w=None),
               dict(out=None), dict(ws=None), dict(q=FAKE + 8), dict(pool=FAKE + 8), dict(w=FAKE + 8),
               dict(out=FAKE + 8), dict(ws=FAKE + 8), dict(B=0), dict(T=-1), dict(bt_stride=0), dict(keys=-1),
               dict(opts=_opts(mask=-1)), dict(opts=_opts(mask=3)), dict(opts=_opts(mask=2, window=0)),
               dict(opts=_opts(scale=float("nan"))), dict(opts=_opts(scale=float("inf"))),
               dict(opts=_opts(num_splits=-1)),
               # a decode's flags mean nothing here
               dict(opts=_opts(flags=M.MLA_FLAG_KERNEL_TIMING)), dict(opts=_opts(flags=4)), dict(opts=_opts(flags=8)),
               dict(dims=_dims(num_heads=0)), dict(dims=_dims(v_head=0)), dict(dims=_dims(page_size=0))):
        assert _prefill(lib, fmt, **kw) == INVALID, kw
    for kw in (dict(num_heads=129), dict(kv_lora_rank=576), dict(kv_lora_rank=32), dict(kv_lora_rank=96),
               dict(qk_nope=136), dict(qk_nope=100), dict(qk_rope=72), dict(qk_rope=12), dict(v_head=136),
               dict(v_head=100), dict(page_size=1 << 20, num_pages=1 << 12)):
        assert _prefill(lib, fmt, dims=_dims(**kw)) == UNSUPPORTED, kw
    for kw in (dict(keys=(1 << 28) + 1), dict(T=(1 << 28) + 1), dict(B=(1 << 20) + 1), dict(opts=_opts(num_splits=257))):
        assert _prefill(lib, fmt, **kw) == UNSUPPORTED, kw
    assert _prefill(lib, fmt, ws_bytes=4096) == TOO_SMALL


def test_prefill_fp8_wants_its_scales(lib):
    assert _prefill(lib, M.MLA_CACHE_E4M3, scales=None) == INVALID
    assert _prefill(lib, M.MLA_CACHE_E4M3, w_scale=None) == INVALID


def test_prefill_workspace_size(lib):
    def size(fmt=0, B=2, T=1000, keys=1000, **kw):
        dims = _dims(**{k: kw.pop(k) for k in list(kw) if k in ("num_heads", "kv_lora_rank")})
        return M.mla_prefill_workspace_size(dims, _opts(**{"num_splits": 1, **kw}), fmt, B, T, keys)
    a = size()
    # every head's keys and values (128 + 128 values of 2 bytes a row; the rope part is the heads' own row's)
    assert a >= 1000 * 256 * 2 * 128
    assert size(keys=2000) > a and size(num_splits=2) > a and size(T=0, keys=0) > 0
    assert size(fmt=M.MLA_CACHE_E4M3) > a          # the widened weights
    # beyond 4 GiB of keys and values the heads go in passes: no more than that, and the rows themselves
    keys = 1 << 20
    big = size(B=1, T=1024, keys=keys)
    assert big < (4 << 30) + keys * 2 * 576 + (1 << 30)
    n = ctypes.c_size_t()
    for rc, fmt, out in ((INVALID, 3, ctypes.byref(n)), (INVALID, -1, ctypes.byref(n)), (INVALID, 0, None)):
        assert lib.mla_prefill_workspace_size(ctypes.byref(_dims()), ctypes.byref(_opts()), fmt, 2, 2, 10, out) == rc
    with pytest.raises(M.MlaError):
        size(num_heads=0)


def test_row_bytes():
    assert [M.mla_cache_row_bytes(f, 512, 64) for f in (0, 1, 2)] == [1152, 640, 400]
    assert M.mla_cache_row_bytes(M.MLA_CACHE_E2M1, 64, 32) == 48 + 64     # 32 + 2 bytes, zeros up to 48
    with pytest.raises(ValueError):
        M.mla_cache_row_bytes(3, 512, 64)


def test_wrappers_refuse_cpu_tensors_and_shapes_that_disagree():
    bf = dict(dtype=torch.bfloat16)
    off, table, lens = (torch.tensor([0, 1], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32),
                        torch.ones(1, dtype=torch.int32))
    new, gamma, freqs = torch.zeros(1, 576, **bf), torch.ones(512, **bf), torch.zeros(8, 64, **bf)
    pool, q = torch.zeros(1, 64, 576, **bf), torch.zeros(1, 4, 192, **bf)
    kw = dict(page_size=64, epsilon=1e-6)
    with pytest.raises(TypeError):
        M.mla_cache_append(new, off, pool, table, lens, freqs, gamma, **kw)          # on the CPU
    with pytest.raises(ValueError):
        M.mla_cache_append(new[:, :570], off, pool, table, lens, freqs, gamma, **kw)
    wk, wv = torch.zeros(4, 512, 128, **bf), torch.zeros(4, 128, 512, **bf)
    for fn, extra in ((M.mla_prefill_paged, dict(total_keys=1)), (M.mla_prefill_paged_fp4, dict(total_keys=1)),
                      (M.mla_decode_paged_fp4, {})):
        with pytest.raises(ValueError):
            fn(q, off, pool, table, lens, wk, wv, page_size=64, **extra)              # on the CPU
        with pytest.raises(ValueError):
            fn(q, off, pool, table, lens, wk[:3], wv, page_size=64, **extra)


@pytest.mark.parametrize("fmt", [R.E4M3, R.E2M1])
def test_reference_formats_round_to_the_nearest_code(fmt):
    """The reference that the GPU tests compare bits with, against the formats' definition."""
    rng = np.random.default_rng(7)
    y = R.bf16_bits(rng.standard_normal((64, 512)) * np.exp(4 * rng.standard_normal((64, 1))))
    rows, scales = R.encode(y, np.zeros((64, 64), np.uint16), fmt)
    assert rows.shape[1] == M.mla_cache_row_bytes(fmt, 512, 64)
    grid, limit, group = (R.e4m3_grid(), 448.0, 512) if fmt == R.E4M3 else (R.E2M1_GRID, 7.0, 32)
    if fmt == R.E4M3:
        scale = scales.astype(np.float64)[:, None]
    else:
        scale = np.ldexp(1.0, rows[:, 256:272].astype(int) - 127).reshape(-1, 1)
    got = R.decode(rows, scales, fmt, 512, 64)[:, :512].reshape(-1, group)
    want = R.bf16_values(y).reshape(-1, group)
    top = np.abs(want).max(1, keepdims=True)
    assert (top <= limit * scale).all() and (top > limit * scale / 2).all()      # the least power of two
    best = np.abs(np.abs(want / scale)[..., None] - grid).min(-1)
    assert np.array_equal(np.abs(got / scale - want / scale), best)             # the nearest code, exactly
    assert (got * want >= 0).all()


def test_reference_rounds_to_bf16_as_torch_does():
    x = np.random.default_rng(3).standard_normal(100000) * np.exp(np.linspace(-80, 80, 100000))
    want = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(R.bf16_bits(x.astype(np.float32)), want)
