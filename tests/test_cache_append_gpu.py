"""GPU: mla_cache_append (new latent rows into a bf16, e4m3 or e2m1 cache) against plain
64-bit numpy forms, bit for bit.

Each stored value is a rounding of an exactly defined real number (RMSNorm and rotation
rounded once to bf16, codes of the bf16 value over a power of two), so there is no tolerance:
pools, row scales, turned queries and returned rows are compared bitwise, rows that no token
owns included.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-6))
WIDE, NARROW = dict(N=128, R=64, L=512), dict(N=32, R=16, L=64)
FORMATS = {"bf16": ref.BF16, "e4m3": ref.E4M3, "e2m1": ref.E2M1}


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
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def same(a, b):
    """Equal bf16 bits; any NaN equals any NaN."""
    nan = (a & 0x7FFF) > 0x7F80
    return np.array_equal(nan, (b & 0x7FFF) > 0x7F80) and np.array_equal(a[~nan], b[~nan])


class Case:
    """Seeded requests: tables over a pool of random bytes, new rows, queries, the expected result."""

    def __init__(self, fmt, seed=1, *, N, R, L, H=3, ps=16, qlens=(1,), past=(0,), new=None, gamma=None, eps=EPS,
                 pad=0):
        r = np.random.default_rng(seed)
        B, self.T = len(qlens), int(sum(qlens))
        self.N, self.R, self.L, self.H, self.ps, self.fmt, self.eps = N, R, L, H, ps, fmt, eps
        self.lens = np.array([a + b for a, b in zip(qlens, past)], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        pages = -(-self.lens // ps)
        order = r.permutation(int(pages.sum()) + 2).astype(np.int32)
        self.table = np.full((B, max(1, int(pages.max()))), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        rows = len(order) * ps
        width = {ref.BF16: 2 * (L + R), ref.E4M3: L + 2 * R,
                 ref.E2M1: -(-(L // 2 + L // 32) // 16) * 16 + 2 * R}[fmt]
        self.pool = r.integers(0, 256, (rows, width), np.uint8)
        self.scales = r.random(rows, np.float32) if fmt == ref.E4M3 else None
        Tp = self.T + pad
        self.new = ref.bf16_bits(r.standard_normal((Tp, L + R)) * np.exp2(r.integers(-3, 4, (Tp, 1)))) if new is None else new
        self.q = ref.bf16_bits(r.standard_normal((Tp, H, N + R)))
        self.gamma = ref.bf16_bits(1 + 0.3 * r.standard_normal(L)) if gamma is None else gamma
        ang = np.arange(int(self.lens.max()))[:, None] * 10000.0 ** (-2 * np.arange(R // 2) / R)
        self.freqs = ref.bf16_bits(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(len(ang), R))
        req = np.repeat(np.arange(B), qlens)
        self.pos = np.concatenate([np.arange(n - k, n) for k, n in zip(qlens, self.lens)]).astype(np.int64)
        self.row = self.table[req, self.pos // ps].astype(np.int64) * ps + self.pos % ps

    def expected(self):
        T = self.T
        y, rope, q = ref.append(self.new[:T], self.gamma, self.freqs, self.pos, self.eps, self.L, self.R, self.q[:T],
                                self.N)
        rows, scales = ref.encode(y, rope, self.fmt)
        pool = self.pool.copy()
        pool[self.row] = rows
        all_scales = None
        if scales is not None:
            all_scales = self.scales.copy()
            all_scales[self.row] = scales
        return pool, all_scales, q, ref.bf16_bits(ref.decode(rows, scales, self.fmt, self.L, self.R))

    def args(self, dev):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        return dict(kv_new=bf16(self.new, dev), input_row_offsets=t(self.offsets), kv_pool=t(self.pool),
                    block_table=t(self.table), cache_lens=t(self.lens), freqs_cis=bf16(self.freqs, dev),
                    kv_norm_gamma=bf16(self.gamma, dev), page_size=self.ps, epsilon=self.eps, cache_format=self.fmt,
                    kv_scales=None if self.scales is None else t(self.scales), q=bf16(self.q, dev))


def run(c, dev, q="out", rows=True, debug=True, **over):
    import mla_decode_attention_06_gb300 as M
    a = c.args(dev)
    a.update(over)
    given = a["q"]
    q_out = torch.full_like(given, float("nan")) if q == "out" else None
    if q is None:
        a["q"] = None
    rows_out = torch.full((len(c.new), c.L + c.R), float("nan"), dtype=torch.bfloat16, device=dev) if rows else None
    M.mla_cache_append(**a, q_out=q_out, rows_out=rows_out, debug=debug)
    torch.cuda.synchronize()
    return a, (q_out if q == "out" else given), rows_out


def check(c, dev, **kw):
    a, q, rows_out = run(c, dev, **kw)
    pool, scales, q_ref, rows = c.expected()
    if c.fmt == ref.BF16:
        assert same(a["kv_pool"].cpu().numpy().view(np.uint16), pool.view(np.uint16))
    else:
        assert np.array_equal(a["kv_pool"].cpu().numpy(), pool)
    if scales is not None:
        assert np.array_equal(a["kv_scales"].cpu().numpy().view(np.uint32), scales.view(np.uint32))
    if kw.get("q", "out") is not None:
        assert same(bits(q)[:c.T], q_ref)
        assert not np.array_equal(q_ref, c.q[:c.T]) or int(c.pos.max()) == 0
    else:
        assert np.array_equal(bits(q), c.q)
    if rows_out is not None:
        assert same(bits(rows_out)[:c.T], rows)
    return a, q, rows_out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", ["wide", "narrow"])
@pytest.mark.parametrize("requests", [((1,), (0,)), ((1,), (70,)), ((3, 1, 20), (0, 15, 16)), ((1,) * 40, tuple(range(40)))])
def test_bitwise(dev, fmt, shape, requests):
    c = Case(FORMATS[fmt], **(WIDE if shape == "wide" else NARROW), qlens=requests[0], past=requests[1])
    check(c, dev)


@pytest.mark.parametrize("heads", [1, 43, 128])
@pytest.mark.parametrize("q", ["out", "in place", None])
def test_queries(dev, heads, q):
    # 43 heads of 24 pieces: the last block of a token is not full
    check(Case(ref.E2M1, 2, **WIDE, H=heads, qlens=(2, 5), past=(9, 0)), dev, q=q)


@pytest.mark.parametrize("widths", [dict(N=0, R=8, L=32), dict(N=8, R=128, L=480), dict(N=64, R=72, L=96)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_odd_widths(dev, fmt, widths):
    check(Case(FORMATS[fmt], 3, **widths, qlens=(4, 3), past=(1, 30)), dev)


def test_many_requests(dev):
    # 1,500 requests: the request of a token takes three rounds of probes; some have no token
    r = np.random.default_rng(4)
    qlens = r.integers(0, 3, 1500)
    qlens[-1] = 1
    check(Case(ref.E4M3, 4, **NARROW, qlens=tuple(qlens), past=tuple(r.integers(0, 20, 1500))), dev)


@pytest.mark.parametrize("fmt", FORMATS)
def test_strided_rows_and_pages(dev, fmt):
    # the new rows as a slice of a wider projection, pages of 1 and of 128 rows
    for ps in (1, 128):
        c = Case(FORMATS[fmt], 5, **WIDE, ps=ps, qlens=(7, 2), past=(130, 0))
        wide = torch.full((c.T, 1536 + 576 + 8), float("nan"), dtype=torch.bfloat16, device=dev)
        wide[:, 1536:1536 + 576] = bf16(c.new, dev)
        check(c, dev, kv_new=wide[:, 1536:1536 + 576])


@pytest.mark.parametrize("fmt", FORMATS)
def test_extreme_rows(dev, fmt):
    # zeros of both signs, one large value, subnormals, the largest bf16, spans of 2^+-60,
    # values past the fp32 path's range, NaN and infinity; gamma of every size
    L, R = 64, 16
    r = np.random.default_rng(6)
    x = r.standard_normal((12, L + R))
    x[0] = 0
    x[1, :L] = -0.0
    x[2, :L] = 0
    x[2, 5] = 3.0
    x[3] *= 2.0 ** -130
    x[4] *= 2.0 ** 120
    x[5] *= np.exp2(r.integers(-60, 60, L + R))
    x[6] *= 2.0 ** -45
    x[7] *= 2.0 ** 70
    x[8, 3] = np.nan
    x[9, 40] = np.inf
    x[10] *= 2.0 ** 56
    gamma = r.standard_normal(L)
    gamma[:6] = [0, -0.0, 2.0 ** 100, 2.0 ** -100, -7.0, 2.0 ** -133]
    for eps in (EPS, 1e30):
        check(Case(FORMATS[fmt], 6, N=32, R=R, L=L, qlens=(12,), past=(3,), new=ref.bf16_bits(x),
                   gamma=ref.bf16_bits(gamma), eps=float(np.float32(eps))), dev)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_code_borders(dev, fmt):
    # RMSNorm of a row with mean square 1 - eps keeps its values, so the codes see exactly the
    # ties and the largest magnitudes that the scale rule names: rows of +-1 times gamma
    L, R = 64, 16
    new = np.ones((4, L + R))
    new[1::2, ::3] = -1
    grid = ref.E2M1_GRID if fmt == "e2m1" else ref.e4m3_grid()[60:]
    mids = (grid[1:] + grid[:-1]) / 2
    for top in (448.0, 449.0, 7.0, 7.0625, 6.0, 6.03125, 1.75, 1.7578125):
        g = np.resize(np.concatenate([mids, grid]), L)
        g = np.where(g > top, 0.25, g)
        g[[0, 32]] = top
        c = Case(FORMATS[fmt], 7, N=32, R=R, L=L, qlens=(4,), past=(0,), new=ref.bf16_bits(new),
                 gamma=ref.bf16_bits(g), eps=0.0)
        check(c, dev)


def test_equals_scatter_and_prologue(dev):
    # a bf16 cache: writing the raw rows and running the branch prologue gives the same bits
    import mla_decode_attention_06_gb300 as M
    c = Case(ref.BF16, 8, **WIDE, H=16, qlens=(1, 4, 2, 300), past=(0, 7, 64, 20))
    a, q, _ = run(c, dev)
    b = c.args(dev)
    pool = b["kv_pool"].clone()
    pool[torch.from_numpy(c.row).to(dev)] = b["kv_new"].view(torch.uint8).view(c.T, -1)
    M.mla_branch_prologue(b["q"], b["input_row_offsets"], pool, b["block_table"], b["cache_lens"], b["freqs_cis"],
                          b["kv_norm_gamma"], page_size=c.ps, kv_lora_rank=c.L, epsilon=c.eps)
    assert torch.equal(pool[torch.from_numpy(c.row).to(dev)], a["kv_pool"][torch.from_numpy(c.row).to(dev)])
    assert np.array_equal(bits(b["q"]), bits(q))


@pytest.mark.parametrize("q", ["out", "in place"])
def test_padding_tokens_are_left_alone(dev, q):
    c = Case(ref.E4M3, 9, **NARROW, qlens=(2, 1), past=(5, 0), pad=6)
    _, got, rows = check(c, dev, q=q)
    if q == "out":
        assert torch.isnan(got[c.T:].float()).all()
    else:
        assert np.array_equal(bits(got)[c.T:], c.q[c.T:])
    assert torch.isnan(rows[c.T:].float()).all()


def test_bad_tokens_are_skipped_and_reported(dev):
    import mla_decode_attention_06_gb300 as M
    for what in ("page", "high page", "table", "negative"):
        c = Case(ref.E2M1, 10, **NARROW, qlens=(2, 2), past=(0, 30))
        pool, _, q_ref, _ = c.expected()
        a = c.args(dev)
        bad = np.array([False, False, True, True])
        if what == "page":
            a["block_table"][1, 1] = -7
        elif what == "high page":
            a["block_table"][1, 1] = len(c.pool) // c.ps
        elif what == "table":
            a["freqs_cis"] = a["freqs_cis"][:31].contiguous()     # positions 30 and 31: the second is past it
            bad = np.array([False, False, False, True])
        else:
            a["cache_lens"][1] = 1                                 # two tokens, one cached: positions -1 and 0
            bad = np.array([False, False, True, False])
        q_out, before = torch.zeros_like(a["q"]), c.pool.copy()
        with pytest.raises(M.MlaError) as e:
            M.mla_cache_append(**a, q_out=q_out, debug=True)
        assert e.value.code == 5
        got = a["kv_pool"].cpu().numpy()
        for t in range(4):
            if what == "negative" and t == 3:
                continue                                           # written, at another position
            assert np.array_equal(got[c.row[t]], (before if bad[t] else pool)[c.row[t]])
            assert np.array_equal(bits(q_out)[t], np.zeros_like(q_ref[t]) if bad[t] else q_ref[t])


def test_no_tokens(dev):
    c = Case(ref.BF16, 11, **NARROW, qlens=(1,), past=(4,))
    a = c.args(dev)
    import mla_decode_attention_06_gb300 as M
    a["kv_new"], a["q"] = a["kv_new"][:0], a["q"][:0]
    a["input_row_offsets"][:] = 0
    M.mla_cache_append(**a, debug=True)
    assert np.array_equal(a["kv_pool"].cpu().numpy(), c.pool)


def test_captured_and_replayed(dev):
    import mla_decode_attention_06_gb300 as M
    c = Case(ref.E2M1, 12, **WIDE, H=16, qlens=(1, 1, 1), past=(3, 100, 0))
    a = c.args(dev)
    a["q_out"], a["workspace"] = torch.empty_like(a["q"]), torch.empty(256, dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        M.mla_cache_append(**a)
    d = Case(ref.E2M1, 13, **WIDE, H=16, qlens=(1, 1, 1), past=(3, 100, 0))
    a["kv_new"].copy_(bf16(d.new, dev))
    a["q"].copy_(bf16(d.q, dev))
    g.replay()
    torch.cuda.synchronize()
    c.new, c.q = d.new, d.q
    pool, _, q_ref, _ = c.expected()
    assert np.array_equal(a["kv_pool"].cpu().numpy(), pool)
    assert np.array_equal(bits(a["q_out"]), q_ref)


def exact_bf16(v):
    """A Fraction's bf16 bits (nearest, ties to even); the sign of a zero is not asked."""
    a = abs(v)
    if a == 0:
        return 0
    e = max(a.numerator.bit_length() - a.denominator.bit_length(), -126)
    while Fraction(2) ** e > a and e > -126:
        e -= 1
    n = round(a / Fraction(2) ** (e - 7))
    mag = min((e + 1 + 127 << 7) if n >= 256 else ((e + 127 << 7) + n - 128 if n >= 128 else n), 0x7F80)
    return mag | (0x8000 if v < 0 else 0)


def test_rotations_past_the_normal_range(dev):
    # products below 2^-126 and past 2^128, sums of either size: each result is the exact value
    # rounded once, in the append and in the prologue
    import mla_decode_attention_06_gb300 as M
    r = np.random.default_rng(51)
    c = Case(ref.BF16, 14, **NARROW, H=16, qlens=(12,), past=(0,))
    wild = lambda shape, lo, hi: ref.bf16_bits(r.choice([-1, 1], shape) * (1 + r.integers(0, 128, shape) / 128) *  # noqa: E731
                                               np.exp2(r.integers(lo, hi, shape)))
    c.q[..., c.N:] = wild(c.q[..., c.N:].shape, -133, 128)
    c.new[:, c.L:] = wild(c.new[:, c.L:].shape, -133, 128)
    c.freqs = wild(c.freqs.shape, -60, 2)
    # halfway between two bf16 values but for a product of 2^-150
    tie = ref.bf16_bits(np.array([1.5 * 2.0 ** -100, 2.0 ** -130]))
    c.q[0, :, c.N:c.N + 2] = c.new[0, c.L:c.L + 2] = tie
    c.freqs[0, :2] = ref.bf16_bits(np.array([1 + 2.0 ** -7, 2.0 ** -20]))
    c.q[1, :, c.N:c.N + 2] = c.new[1, c.L:c.L + 2] = tie
    c.freqs[1, :2] = ref.bf16_bits(np.array([1 + 2.0 ** -7, -2.0 ** -20]))

    def turned(x, pos):
        v = np.vectorize(lambda b: Fraction(float(ref.bf16_values(b))), otypes=[object])
        x, f = v(x), v(c.freqs[pos])
        out = np.empty(x.shape, np.uint16)
        for i in range(0, x.shape[-1], 2):
            x0, x1, cos, sin = x[..., i], x[..., i + 1], f[i], f[i + 1]
            out[..., i] = np.vectorize(exact_bf16, otypes=[np.uint16])(x0 * cos - x1 * sin)
            out[..., i + 1] = np.vectorize(exact_bf16, otypes=[np.uint16])(x0 * sin + x1 * cos)
        return out

    _, q, rows = run(c, dev)
    b = c.args(dev)
    pool = b["kv_pool"].clone()
    at = torch.from_numpy(c.row).to(dev)
    pool[at] = b["kv_new"].view(torch.uint8).view(c.T, -1)
    M.mla_branch_prologue(b["q"], b["input_row_offsets"], pool, b["block_table"], b["cache_lens"], b["freqs_cis"],
                          b["kv_norm_gamma"], page_size=c.ps, kv_lora_rank=c.L, epsilon=c.eps)
    pro_rows = pool[at].cpu().numpy().view(np.uint16)
    no_sign = lambda x: np.where(x & 0x7FFF, x, 0)  # noqa: E731
    for t in range(c.T):
        want_q, want_r = turned(c.q[t, :, c.N:], t), turned(c.new[t, c.L:], t)
        for got_q, got_r in ((bits(q)[t, :, c.N:], bits(rows)[t, c.L:]), (bits(b["q"])[t, :, c.N:], pro_rows[t, c.L:])):
            assert np.array_equal(no_sign(got_q), no_sign(want_q)) and np.array_equal(no_sign(got_r), no_sign(want_r)), t
