"""CPU-side checks of the operators over 8-bit codes (mla_rmsnorm_quant, mla_linear_fp8, mla_linear_int8,
mla_indexer_append) and of mla_cache_read: what they refuse before anything reaches a GPU, and their
reference's formats."""
import ctypes

import numpy as np
import pytest
import torch

import code_ref as cr
import latent_ref as ref
import mla_decode_attention_06_gb300 as M

FAKE = 0x10000   # aligned, never dereferenced: every case below fails validation first
INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 3
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from mla_decode_attention_06_gb300 import _lib, build
    build.build()
    return _lib.load()


def _norm(lib, fmt=1, rows=2, width=512, x=FAKE, stride=512, res=FAKE, res_out=FAKE, gamma=FAKE, eps=1e-6, y=None,
          codes=FAKE, scales=FAKE):
    return lib.mla_rmsnorm_quant(fmt, rows, width, x, stride, res, res_out, gamma, eps, y, codes, scales, None)


def test_norm_refusals(lib):
    for kw in (dict(fmt=-1), dict(fmt=3), dict(rows=-1), dict(width=0), dict(stride=504), dict(stride=516), dict(eps=-1.0),
               dict(eps=NAN), dict(eps=INF), dict(x=None), dict(res=None), dict(res_out=None), dict(codes=None),
               dict(scales=None), dict(fmt=0, y=FAKE), dict(fmt=0, y=FAKE, codes=None), dict(fmt=0, codes=None, scales=None),
               dict(x=FAKE + 8), dict(res=FAKE + 8), dict(res_out=FAKE + 8), dict(gamma=FAKE + 8), dict(y=FAKE + 8),
               dict(codes=FAKE + 8)):
        assert _norm(lib, **kw) == INVALID, kw
    for kw in (dict(width=508, stride=512), dict(width=32776, stride=32776)):
        assert _norm(lib, **kw) == UNSUPPORTED, kw


@pytest.mark.parametrize("name", ["mla_linear_fp8", "mla_linear_int8"])
def test_linear_refusals(lib, name):
    def call(T=2, n=64, k=64, x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, out=FAKE, stride=64, flags=0, wsp=FAKE, wsp_bytes=256):
        return getattr(lib, name)(T, n, k, x, xs, w, ws, out, stride, flags, wsp, wsp_bytes, None)
    for kw in (dict(T=-1), dict(n=0), dict(k=0), dict(stride=56), dict(flags=2), dict(x=None), dict(xs=None), dict(w=None),
               dict(ws=None), dict(out=None), dict(wsp=None), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(ws=FAKE + 4),
               dict(out=FAKE + 8)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(n=60), dict(k=72), dict(stride=68), dict(T=(1 << 22) + 1), dict(n=(1 << 24) + 8, stride=1 << 25),
               dict(k=(1 << 24) + 16), dict(k=(1 << 31) - 16)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(wsp_bytes=255), dict(wsp=FAKE + 8)):
        assert call(**kw) == TOO_SMALL, kw


def _dims(**kw):
    d = dict(num_heads=1, qk_nope=0, qk_rope=64, kv_lora_rank=512, v_head=1, page_size=64, num_pages=100)
    d.update(kw)
    return M.MlaDims(**d)


def test_read_refusals(lib):
    def call(dims=None, fmt=0, off=FAKE, B=2, T=2, pool=FAKE, scales=None, table=FAKE, bt_stride=4, lens=FAKE, out=FAKE,
             flags=0, ws=FAKE, ws_bytes=256):
        return lib.mla_cache_read(ctypes.byref(dims or _dims()), fmt, off, B, T, pool, scales, table, bt_stride, lens, out,
                                  flags, ws, ws_bytes, None)
    for kw in (dict(fmt=-1), dict(fmt=3), dict(off=None), dict(B=0), dict(T=-1), dict(pool=None), dict(table=None),
               dict(bt_stride=0), dict(lens=None), dict(out=None), dict(flags=2), dict(ws=None), dict(scales=FAKE),
               dict(fmt=1), dict(fmt=2, scales=FAKE), dict(pool=FAKE + 8), dict(out=FAKE + 8),
               dict(dims=_dims(qk_rope=0)), dict(dims=_dims(kv_lora_rank=0)), dict(dims=_dims(page_size=0)),
               dict(dims=_dims(num_pages=0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(kv_lora_rank=544), dict(kv_lora_rank=48), dict(qk_rope=136), dict(qk_rope=12),
               dict(page_size=1 << 20, num_pages=1 << 12)):
        assert call(dims=_dims(**kw)) == UNSUPPORTED, kw
    assert call(ws_bytes=0) == TOO_SMALL and call(ws=FAKE + 8) == TOO_SMALL
    assert lib.mla_cache_read(None, 0, FAKE, 2, 2, FAKE, None, FAKE, 4, FAKE, FAKE, 0, FAKE, 256, None) == INVALID


def test_indexer_append_refusals(lib):
    def call(H=4, D=128, R=64, ps=64, pages=10, k=FAKE, stride=128, off=FAKE, B=2, T=2, q=FAKE, weight=FAKE, codes=FAKE,
             scales=FAKE, cache=FAKE, k_scales=FAKE, table=FAKE, bt_stride=4, lens=FAKE, freqs=FAKE, max_len=64, gamma=FAKE,
             beta=FAKE, eps=1e-6, flags=0, ws=FAKE, ws_bytes=256):
        return lib.mla_indexer_append(H, D, R, ps, pages, k, stride, off, B, T, q, weight, codes, scales, cache, k_scales,
                                      table, bt_stride, lens, freqs, max_len, gamma, beta, eps, flags, ws, ws_bytes, None)
    no_q = dict(q=None, weight=None, codes=None, scales=None)
    for kw in (dict(H=0), dict(D=0), dict(R=0), dict(R=136), dict(ps=0), dict(pages=0), dict(k=None), dict(stride=120),
               dict(stride=132), dict(off=None), dict(B=0), dict(T=-1), dict(q=None), dict(codes=None), dict(scales=None),
               dict(no_q, weight=FAKE), dict(cache=None), dict(k_scales=None), dict(table=None), dict(bt_stride=0),
               dict(lens=None), dict(max_len=0), dict(gamma=None), dict(beta=None), dict(eps=-1.0), dict(eps=NAN),
               dict(eps=INF), dict(flags=2), dict(ws=None), dict(k=FAKE + 8), dict(q=FAKE + 8), dict(codes=FAKE + 8),
               dict(cache=FAKE + 8), dict(freqs=FAKE + 8), dict(gamma=FAKE + 8), dict(beta=FAKE + 8)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=132, stride=136, R=64), dict(D=264, stride=264), dict(R=60), dict(ps=1 << 20, pages=1 << 12),
               dict(T=1 << 30, H=1 << 20), dict(T=(1 << 31) - 40, H=1)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(ws_bytes=0) == TOO_SMALL and call(ws=FAKE + 8) == TOO_SMALL
    # without queries the head count is not looked at, without rotations the rope width
    assert call(H=0, ws_bytes=0, **no_q) == TOO_SMALL and call(freqs=None, R=-3, max_len=0, ws_bytes=0) == TOO_SMALL


def test_wrappers_refuse_shapes_types_and_cpu_tensors():
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    x = torch.zeros(2, 64, **bf)
    for bad in (lambda: M.mla_rmsnorm_quant(x),                                      # on the CPU
                lambda: M.mla_rmsnorm_quant(x[0]), lambda: M.mla_rmsnorm_quant(x, code_format=7),
                lambda: M.mla_rmsnorm_quant(x, residual_out=x), lambda: M.mla_rmsnorm_quant(x.float())):
        with pytest.raises((TypeError, ValueError)):
            bad()
    c, s = torch.zeros(2, 64, dtype=torch.int8), torch.ones(2)
    for bad in (lambda: M.mla_linear_int8(c, s, c, s), lambda: M.mla_linear_int8(c, s, c[:, :32], s),
                lambda: M.mla_linear_int8(c, s[:1], c, s), lambda: M.mla_linear_int8(c, s, c, s[:1]),
                lambda: M.mla_linear_fp8(c, s, c, s)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    off, table, lens = torch.tensor([0, 2], **i32), torch.zeros(1, 1, **i32), torch.ones(1, **i32)
    pool = torch.zeros(1, 64, 576, **bf)
    for bad in (lambda: M.mla_cache_read(off, pool, table, lens, kv_lora_rank=512, qk_rope=64, page_size=64, total_rows=2),
                lambda: M.mla_cache_read(off, pool, table, lens, kv_lora_rank=512, qk_rope=64, page_size=60, total_rows=2)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    kc, ks, k = torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64), torch.zeros(2, 64, **bf)
    for kw in ({}, dict(q=torch.zeros(2, 3, 32, **bf)), dict(q_weight=s), dict(k_norm_gamma=k[0, :8])):
        with pytest.raises((TypeError, ValueError)):
            M.mla_indexer_append(k, off, kc, ks, table, lens, page_size=64, **kw)


def test_reference_codes_are_the_nearest():
    r = np.random.default_rng(3)
    y = ref.bf16_bits(r.standard_normal((40, 256)) * np.exp(3 * r.standard_normal((40, 1))))
    want = ref.bf16_values(y)
    codes, scale = cr.encode(y, cr.INT8)
    q = want / scale.astype(np.float64)[:, None]
    assert np.abs(codes.view(np.int8)).max() <= 127 and (np.abs(codes.view(np.int8)).max(1) == 127).all()
    assert (np.abs(codes.view(np.int8) - q) <= 0.5).all()
    codes, scale = cr.encode(y, cr.E4M3)
    q, got = want / scale.astype(np.float64)[:, None], cr.E4M3_VALUES[codes]
    best = np.abs(np.abs(q)[..., None] - ref.e4m3_grid()).min(-1)
    assert np.array_equal(np.abs(got - q), best)
    top = np.abs(want).max(1)
    assert (top <= 448 * scale).all() and (top > 224 * scale).all()
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, t)
