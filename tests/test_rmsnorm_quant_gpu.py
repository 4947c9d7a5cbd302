"""GPU: mla_rmsnorm_quant (residual addition, RMSNorm, e4m3 or int8 codes) against plain 64-bit
numpy forms, bit for bit.

Every output is a rounding of an exactly defined real number (the sum, the normalised row, the
quotient of a bf16 value and its scale), so there is no tolerance."""
import numpy as np
import pytest
import torch

import code_ref as cr
import latent_ref as ref

pytestmark = pytest.mark.gpu
EPS = float(np.float32(1e-6))
FORMATS = {"bf16": cr.NONE, "e4m3": cr.E4M3, "int8": cr.INT8}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_decode_attention_06_gb300 import build
    build.build()
    return torch.device("cuda:0")


def bf16(bits, dev):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(dev).view(torch.bfloat16)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def same(a, b):
    """Equal bf16 bits; any NaN equals any NaN."""
    nan = (a & 0x7FFF) > 0x7F80
    return np.array_equal(nan, (b & 0x7FFF) > 0x7F80) and np.array_equal(a[~nan], b[~nan])


def check(dev, fmt, x, residual=None, gamma=None, eps=EPS, pad=0, in_place=False, y_out=True):
    import mla_decode_attention_06_gb300 as M
    T, D = x.shape
    wide = torch.full((T, D + pad), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, :D] = bf16(x, dev)
    r = None if residual is None else bf16(residual, dev)
    r_out = None if r is None or in_place else torch.full_like(r, float("nan"))
    y = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=dev) if y_out else None
    got, scales, h = M.mla_rmsnorm_quant(wide[:, :D], None if gamma is None else bf16(gamma, dev), epsilon=eps,
                                         code_format=fmt, residual=r, residual_out=r_out, y_out=y)
    h_ref, y_ref = cr.rmsnorm(x, residual, gamma, eps)
    if r is None:
        assert h is None
    else:
        assert h is (r if in_place else r_out) and same(bits(h), h_ref)
        assert in_place or same(bits(r), residual)
    if y_out:
        assert same(bits(y), y_ref)
    if fmt == cr.NONE:
        assert scales is None and same(bits(got), y_ref)
        return
    codes, s = cr.encode(y_ref, fmt)
    assert got.dtype == (torch.float8_e4m3fn if fmt == cr.E4M3 else torch.int8)
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(got.view(torch.uint8).cpu().numpy(), codes)


def rows(seed, T, D, spread=2):
    r = np.random.default_rng(seed)
    return ref.bf16_bits(r.standard_normal((T, D)) * np.exp2(r.integers(-spread, spread + 1, (T, 1))))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [8, 64, 248, 256, 264, 512, 520, 1024, 1032, 1536, 4096, 4104, 8192, 8200, 16384, 32768])
def test_widths(dev, fmt, D):
    """One to four pieces a thread, a row a warp or a block, widths that leave threads without a piece."""
    T = 19 if D <= 1032 else 5
    g = ref.bf16_bits(1 + 0.3 * np.random.default_rng(5).standard_normal(D))
    check(dev, FORMATS[fmt], rows(1, T, D), rows(2, T, D), g)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 7, 8, 9, 700])
@pytest.mark.parametrize("gamma,residual,pad", [(True, False, 576), (False, True, 0), (False, False, 8), (True, True, 24)])
def test_rows_strides_and_parts(dev, fmt, T, gamma, residual, pad):
    for D in (512, 1536):
        g = ref.bf16_bits(1 + 0.3 * np.random.default_rng(5).standard_normal(D)) if gamma else None
        check(dev, FORMATS[fmt], rows(3, T, D), rows(4, T, D) if residual else None, g, pad=pad, y_out=fmt != "int8")


@pytest.mark.parametrize("fmt", FORMATS)
def test_in_place_residual(dev, fmt):
    for D in (256, 2048):
        check(dev, FORMATS[fmt], rows(3, 11, D), rows(4, 11, D), rows(6, 1, D)[0], in_place=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [72, 1304])
@pytest.mark.parametrize("gamma", [True, False])
def test_values_at_the_edges(dev, fmt, D, gamma):
    """Zeros, NaN, infinities, the type's ends, rows far from one, zeros among values, negative zeros."""
    r = np.random.default_rng(8)
    v = r.standard_normal((16, D))
    v[0] = 0.0
    v[1, 5] = np.nan
    v[2, D - 1] = np.inf
    v[3, 0] = -np.inf
    v[4] *= 2.0 ** 124
    v[5] *= 2.0 ** -128
    v[6] = np.where(r.random(D) < 0.5, 2.0 ** -133, 2.0 ** 127)
    v[7] = 2.0 ** -133
    v[8, ::3] = 0.0
    v[9] = -0.0
    v[10] *= np.exp2(r.integers(-60, 60, D))
    v[11] = np.where(r.random(D) < 0.9, 0.0, v[11] * 2.0 ** -70)
    v[12] = 448 * 2.0 ** -6
    v[13] = np.where(r.random(D) < 0.5, 450, -448)
    v[14] *= 2.0 ** -120
    v[15] *= 2.0 ** 60
    x = ref.bf16_bits(v)
    g = None
    if gamma:
        g = ref.bf16_bits(r.standard_normal(D))
        g[3], g[7], g[9] = 0, 0x8000, ref.bf16_bits(np.array(2.0 ** -100))
    check(dev, FORMATS[fmt], x, None, g)
    check(dev, FORMATS[fmt], x, None, g, eps=0.0)
    check(dev, FORMATS[fmt], x, x[::-1].copy(), g)


def test_int8_ties_and_neighbours(dev):
    """Quotients at half-integers (the scale a power of two) and all bf16 values next to them; every bf16
    significand as a row's largest value."""
    D = 512
    half = np.concatenate([np.arange(-63.5, 64), np.arange(-126, 127)])
    x = np.zeros((9, D))
    for i in range(9):
        x[i, :len(half)] = half * 2.0 ** (i - 4)
        x[i, -1] = 127 * 2.0 ** (i - 4)
    check(dev, cr.INT8, ref.bf16_bits(x))
    r = np.random.default_rng(1)
    top = (1 + np.arange(128) / 128)[:, None]
    x = top * r.uniform(-1, 1, (128, 4096))
    x[:, 7] = top[:, 0]
    check(dev, cr.INT8, ref.bf16_bits(x))


def test_e4m3_scale_at_its_steps(dev):
    top = np.array([448, 446, 450, 224, 225, 896, 447.9, 3.5, 3.4921875, 3.515625])[:, None]
    x = top * np.random.default_rng(1).uniform(-1, 1, (10, 640))
    x[:, 3] = top[:, 0]
    check(dev, cr.E4M3, ref.bf16_bits(x))


def test_long_rows_sum_exactly(dev):
    """One value far above the others: a plain fp32 sum would lose most of the row."""
    D = 32768
    v = np.full((3, D), 2.0 ** -11)
    v[:, 17] = [1.0, 3.0, 60.0]
    for fmt in FORMATS.values():
        check(dev, fmt, ref.bf16_bits(v), None, ref.bf16_bits(np.random.default_rng(3).standard_normal(D)))


def test_empty_and_streams_and_graph(dev):
    import mla_decode_attention_06_gb300 as M
    codes, s, h = M.mla_rmsnorm_quant(torch.empty(0, 64, dtype=torch.bfloat16, device=dev))
    assert codes.shape == (0, 64) and s.shape == (0,) and h is None
    x, g = rows(1, 33, 1536), rows(2, 1, 1536)[0]
    want = cr.encode(cr.rmsnorm(x, None, g, EPS)[1], cr.INT8)
    xt, gt = bf16(x, dev), bf16(g, dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    a = M.mla_rmsnorm_quant(xt, gt, epsilon=EPS, code_format=M.MLA_CODES_INT8, stream=side)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = M.mla_rmsnorm_quant(xt, gt, epsilon=EPS, code_format=M.MLA_CODES_INT8)
    for got in (a, b):
        if got is b:
            graph.replay()
        assert np.array_equal(got[0].cpu().numpy().view(np.uint8), want[0])
        assert np.array_equal(got[1].cpu().numpy(), want[1])


def test_offsets_past_32_bits(dev):
    """Rows that lie, and outputs that end, more than 2^31 elements after the first."""
    import mla_decode_attention_06_gb300 as M
    for T, D, stride in ((300, 264, 1 << 23), (66000, 32768, 32768)):
        x = torch.empty((T - 1) * stride + D, dtype=torch.bfloat16, device=dev).as_strided((T, D), (stride, 1))
        last = rows(3, 2, D)
        x.zero_()
        x[-2:] = bf16(last, dev)
        codes, s, _ = M.mla_rmsnorm_quant(x, code_format=M.MLA_CODES_INT8)
        want = cr.encode(last, cr.INT8)
        assert np.array_equal(codes[-2:].cpu().numpy().view(np.uint8), want[0])
        assert np.array_equal(s[-2:].cpu().numpy(), want[1]) and (s[:-2] == 1).all() and not codes[:-2].any()
