"""GPU: mla_prefill_paged (latent attention, expanded form) against a plain 64-bit numpy form, over
bf16, e4m3 and e2m1 caches.

Tolerances, as relative 2-norms over the output.  A rounding to t bits is off by at most
u = eps / 2 of the value and u / sqrt(3) rms at worst (a value at the low end of its binade):
2.3e-3 for bf16, 2.8e-4 for f16.
  f16 sequence: the output's bf16 rounding, V and P in f16, and K in f16, whose share the
  softmax multiplies by the spread of the scores (about 2 here): 2.3e-3 + 4 * 2.8e-4 = 3.4e-3;
  3.5e-3 is asked.  e4m3 calls round latents and weights to f16 too (twice in K, twice in V):
  3.4e-3 + 6 * 2.8e-4 = 5.1e-3.
  bf16 sequence (values that f16 does not hold): (1 + 2 + 2) * 2.3e-3 = 1.2e-2; with e4m3
  (1 + 2 + 2 + 2 + 4) * 2.3e-3 = 2.6e-2.
The log-sum-exp moves by the scores' error: a rounding moves a score of up to 8 by at most
8 * 2^-11 = 3.9e-3 (bf16: 3.1e-2).  K is one, beside it 1.5 of them are left for the sums: 8e-3
(6e-2).  e4m3 calls round the latent and the weight before K, two more: 1.6e-2 (1.25e-1).
"""
import numpy as np
import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

TOL = {"f16": 3.5e-3, "e4m3": 5.1e-3, "bf16": 1.2e-2, "bf16 e4m3": 2.6e-2}
TOL_LSE = {"f16": 8e-3, "e4m3": 1.6e-2, "bf16": 6e-2, "bf16 e4m3": 1.25e-1}
WIDE, NARROW = dict(N=128, R=64, L=512, V=128), dict(N=32, R=16, L=64, V=32)
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


class Case:
    """Seeded requests over a pool whose other rows are NaN in every format (bytes 0xFF)."""

    def __init__(self, fmt="bf16", seed=1, *, N, R, L, V, H=2, ps=16, qlens=(5,), past=(0,), mask=1, window=0,
                 scale=None, pad=0, c=1.0, rope=1.0, w_uv=1.0, q=1.0):
        r = np.random.default_rng(seed)
        self.fmt, self.N, self.R, self.L, self.V, self.H, self.ps = FORMATS[fmt], N, R, L, V, H, ps
        self.mask, self.window, self.T = mask, window, int(sum(qlens))
        self.scale = 1 / np.sqrt(N + R) if scale is None else scale
        B = len(qlens)
        self.lens = np.array([max(0, a + b) for a, b in zip(qlens, past)], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        pages = -(-self.lens // ps)
        self.num_pages = int(pages.sum()) + 2
        order = r.permutation(self.num_pages).astype(np.int32)
        self.table = np.full((B, max(1, int(pages.max()))), -1, np.int32)
        self.values, at = [], 0
        width = {ref.BF16: 2 * (L + R), ref.E4M3: L + 2 * R,
                 ref.E2M1: -(-(L // 2 + L // 32) // 16) * 16 + 2 * R}[self.fmt]
        self.pool = np.full((self.num_pages * ps, width), 0xFF, np.uint8)
        self.scales = np.full(self.num_pages * ps, np.nan, np.float32) if self.fmt == ref.E4M3 else None
        self.rows = []
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
            n = int(self.lens[b])
            j = np.arange(n)
            self.rows.append(self.table[b, j // ps].astype(np.int64) * ps + j % ps)
            x, s = ref.encode(ref.bf16_bits(c * r.standard_normal((n, L))), ref.bf16_bits(rope * r.standard_normal((n, R))),
                              self.fmt)
            self.pool[self.rows[b]] = x
            if s is not None:
                # any fp32 scale is allowed, not only the powers of two that the append writes
                self.scales[self.rows[b]] = s * (1 + 0.3 * r.random(n)).astype(np.float32)
        self.q = ref.bf16_bits(q * r.standard_normal((self.T + pad, H, N + R)))
        uk, uv = r.standard_normal((H, L, N)) / np.sqrt(N), w_uv * r.standard_normal((H, V, L)) / np.sqrt(L)
        if self.fmt == ref.E4M3:
            self.w = [self.coded(uk, r), self.coded(uv, r)]
            self.uk, self.uv = (code * sc.repeat(128, 1)[:, :code.shape[1]].repeat(128, 2)[:, :, :code.shape[2]].astype(np.float64)
                                for code, sc in ((ref_values(x), s) for x, s in self.w))
        else:
            self.w = [ref.bf16_bits(uk), ref.bf16_bits(uv)]
            self.uk, self.uv = (ref.bf16_values(x) for x in self.w)

    @staticmethod
    def coded(w, r):
        na, nb = -(-w.shape[1] // 128), -(-w.shape[2] // 128)
        s = (np.abs(w).max((1, 2))[:, None, None] / 448 * (1 + r.random((len(w), na, nb)))).astype(np.float32)
        full = s.repeat(128, 1)[:, :w.shape[1]].repeat(128, 2)[:, :, :w.shape[2]]
        code = ref.nearest_code(np.abs(w) / full, ref.e4m3_grid()).astype(np.uint8)
        return code | (w < 0).astype(np.uint8) << 7, s

    def cached(self, b):
        return ref.decode(self.pool[self.rows[b]], None if self.scales is None else self.scales[self.rows[b]], self.fmt,
                          self.L, self.R)

    def expected(self):
        with np.errstate(invalid="ignore"):
            return ref.attention(ref.bf16_values(self.q), self.uk, self.uv, [self.cached(b) for b in range(len(self.lens))],
                                 self.lens, self.offsets, self.scale, self.mask, self.window)

    def args(self, dev):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        head = [bf16(self.q, dev), t(self.offsets), t(self.pool)]
        if self.fmt == ref.E4M3:
            head.append(t(self.scales))
        tail = [t(self.table), t(self.lens)]
        for w in self.w:
            tail += [t(w[0]), t(w[1])] if self.fmt == ref.E4M3 else [bf16(w, dev)]
        return head + tail, dict(page_size=self.ps, total_keys=int(self.lens.sum()), scale=float(self.scale), mask=self.mask,
                                 window=self.window)


def ref_values(codes):
    return np.concatenate([ref.e4m3_grid(), [np.nan]])[codes & 127] * np.where(codes >> 7, -1.0, 1.0)


def call(c, dev, args=None, **kw):
    import mla_decode_attention_06_gb300 as M
    a, k = c.args(dev) if args is None else args
    fn = (M.mla_prefill_paged, M.mla_prefill_paged_fp8, M.mla_prefill_paged_fp4)[c.fmt]
    out = torch.full((len(c.q), c.H, c.V), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((len(c.q), c.H), 7.0, device=dev)
    k = dict(dict(k, out=out, lse_out=lse, debug=True), **kw)
    fn(*a, **k)
    torch.cuda.synchronize()
    return out, lse


def compare(c, out, lse, kind):
    want, want_lse = c.expected()
    g, gl = out.float().cpu().numpy().astype(np.float64)[:c.T], lse.cpu().numpy().astype(np.float64)[:c.T]
    want, want_lse = want[:c.T], want_lse[:c.T]
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan) and np.array_equal(np.isnan(gl), np.isnan(want_lse))
    assert (g[want_lse == -np.inf] == 0).all() and np.array_equal(gl == -np.inf, want_lse == -np.inf)
    err = np.linalg.norm((g - want)[~nan]) / max(np.linalg.norm(want[~nan]), 1e-300)
    assert err <= TOL[kind], err
    fin = np.isfinite(want_lse)
    assert not fin.any() or np.abs(gl[fin] - want_lse[fin]).max() <= TOL_LSE[kind]
    return err


def check(c, dev, kind=None, **kw):
    kind = kind or ("e4m3" if c.fmt == ref.E4M3 else "f16")
    out, lse = call(c, dev, **kw)
    compare(c, out, lse, kind)
    assert (out[c.T:] == 7).all() and (lse[c.T:] == 7).all()
    return out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", ["wide", "narrow"])
@pytest.mark.parametrize("qlens,past", [((1,), (0,)), ((128,), (0,)), ((129, 1, 3), (0, 300, 0)), ((257, 40), (100, 5))])
def test_ragged(dev, fmt, shape, qlens, past):
    check(Case(fmt, **(WIDE if shape == "wide" else NARROW), qlens=qlens, past=past), dev)


@pytest.mark.parametrize("n", [2, 64, 127, 255, 256, 300, 511, 520, 700])
def test_lengths(dev, n):
    check(Case(seed=n, **WIDE, H=1, qlens=(n,), past=(0,)), dev)


@pytest.mark.parametrize("mask,window", [(0, 0), (2, 1), (2, 64), (2, 128), (2, 200), (2, 100000)])
def test_masks(dev, mask, window):
    check(Case("e2m1", 3, **WIDE, qlens=(300, 10), past=(45, 400), mask=mask, window=window), dev)


@pytest.mark.parametrize("widths", [dict(N=8, R=8, L=64, V=8), dict(N=72, R=40, L=192, V=120), dict(N=128, R=8, L=448, V=64),
                                    dict(N=64, R=64, L=128, V=128)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_odd_widths(dev, fmt, widths):
    check(Case(fmt, 4, **widths, H=3, ps=8, qlens=(140, 9), past=(3, 150)), dev)


@pytest.mark.parametrize("ps", [1, 7, 64, 512])
def test_page_sizes(dev, ps):
    check(Case("e4m3", 5, **NARROW, ps=ps, qlens=(33, 130), past=(200, 0)), dev)


def test_heads_and_many_requests(dev):
    r = np.random.default_rng(6)
    check(Case("bf16", 6, **NARROW, H=128, qlens=tuple(r.integers(0, 30, 70)), past=tuple(r.integers(0, 90, 70))), dev)


@pytest.mark.parametrize("num_splits", [1, 2, 5, 40])
@pytest.mark.parametrize("mask,window", [(1, 0), (2, 150)])
def test_key_splits(dev, num_splits, mask, window):
    # more splits than a query block has key tiles leaves some of them empty
    check(Case("bf16", 7, **WIDE, qlens=(200, 3), past=(900, 20), mask=mask, window=window, pad=3), dev, num_splits=num_splits)


def test_long_ring(dev):
    # 21 key tiles: the value boxes pass the end of the ring
    check(Case("bf16", 8, **WIDE, H=1, qlens=(260,), past=(2400,)), dev, num_splits=1)


def test_growing_scores(dev):
    # rope columns that grow with the position: every tile raises the running maximum by more
    # than the rescaling threshold
    c = Case("bf16", 9, **WIDE, H=2, qlens=(200,), past=(700,), c=0.5)
    n = int(c.lens[0])
    rope = np.zeros((n, c.R))
    rope[:, 0] = np.arange(n) // 128 * 9.0
    x = ref.bf16_values(c.q)
    x[..., c.N] = 13.0
    c.q = ref.bf16_bits(x)
    c.pool[c.rows[0], -2 * c.R:] = np.ascontiguousarray(ref.bf16_bits(rope)).view(np.uint8)
    out, lse = call(c, dev, num_splits=1)
    want, _ = c.expected()
    g = out.float().cpu().numpy()
    assert np.linalg.norm(g - want) <= TOL["f16"] * np.linalg.norm(want)


def test_empty_rows_and_padding(dev):
    # a request without cache and one with more query tokens than cached ones are reported, as by
    # the decode, and give 0 and -inf where no key is left; tokens of no request keep what they held
    import mla_decode_attention_06_gb300 as M
    c = Case("bf16", 10, **NARROW, qlens=(4, 9, 2), past=(-4, -3, 50), pad=5)
    with pytest.raises(M.MlaError) as e:
        call(c, dev)
    assert e.value.code == 5
    check(c, dev, debug=False)


def test_padding_is_left_alone(dev):
    for splits in (1, 3):
        check(Case("bf16", 10, **NARROW, qlens=(4, 0, 2), past=(0, 0, 50), pad=5), dev, num_splits=splits)


@pytest.mark.parametrize("what", ["c", "small c", "rope", "w_uv", "q", "w_uv down"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_values_that_f16_does_not_hold(dev, fmt, what):
    # magnitudes past f16's range, up or down, take the bf16 sequence; queries need not
    kw = {"c": dict(c=2.0 ** 20, scale=2.0 ** -22), "small c": dict(c=2.0 ** -30, scale=2.0 ** 27, rope=2.0 ** -30),
          "rope": dict(rope=2.0 ** 20, scale=2.0 ** -23), "w_uv": dict(w_uv=2.0 ** 40), "w_uv down": dict(w_uv=2.0 ** -40),
          "q": dict(q=2.0 ** 100, scale=2.0 ** -104)}[what]
    kind = ("e4m3" if fmt == "e4m3" else "f16") if what == "q" else "bf16 e4m3" if fmt == "e4m3" else "bf16"
    c = Case(fmt, 11, **WIDE, qlens=(150, 7), past=(20, 200), **kw)
    check(c, dev, kind)
    if what == "c":
        check(Case(fmt, 11, **WIDE, qlens=(150, 7), past=(20, 200), **kw), dev, kind, num_splits=2)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-30])
def test_scales(dev, scale):
    check(Case("bf16", 12, **NARROW, qlens=(140,), past=(9,), scale=scale), dev)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_nan_and_inf_reach_only_who_sees_them(dev, fmt, bad):
    c = Case(fmt, 13, **NARROW, qlens=(200, 5), past=(0, 60))
    row = c.rows[0][77]
    if fmt == "bf16":
        c.pool[row, 10:12] = np.array([0x7F80 if bad == np.inf else 0x7FC0], np.uint16).view(np.uint8)
    elif fmt == "e4m3":
        c.scales[row] = bad
    else:
        c.pool[row, c.L // 2 + 1] = 0xFF
    out, lse = call(c, dev)
    assert torch.isfinite(out[:77].float()).all() and torch.isfinite(lse[:77]).all()
    assert torch.isnan(out[77:200].float()).all() and torch.isnan(lse[77:200]).all()
    assert torch.isfinite(out[200:].float()).all()
    clean = Case(fmt, 13, **NARROW, qlens=(200, 5), past=(0, 60))
    want, _ = call(clean, dev)
    assert torch.equal(out[:77], want[:77]) and torch.equal(out[200:], want[200:])


def test_head_passes_and_workspace(dev):
    # the same bits whether the heads go through the workspace together or one at a time
    import ctypes
    import mla_decode_attention_06_gb300 as M
    c = Case("bf16", 14, **NARROW, H=5, qlens=(130, 9), past=(7, 300))
    dims = M.MlaDims(num_heads=5, qk_nope=32, qk_rope=16, kv_lora_rank=64, v_head=32, page_size=16, num_pages=c.num_pages)
    opts = M.MlaOpts(mask=1, window=0, scale=float(c.scale), num_splits=1, flags=0)
    n = M.mla_prefill_workspace_size(dims, opts, 0, 2, c.T, int(c.lens.sum()))
    tiles = int(c.lens.sum()) // 128 + 2
    one_head = tiles * 2 * 16384
    want, want_lse = check(c, dev, num_splits=1, workspace=torch.empty(n, dtype=torch.uint8, device=dev))
    for heads in (1, 2, 3):
        ws = torch.empty(n - (5 - heads) * one_head, dtype=torch.uint8, device=dev)
        out, lse = call(c, dev, num_splits=1, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    with pytest.raises(M.MlaError) as e:
        call(c, dev, num_splits=1, workspace=torch.empty(n - 4 * one_head - 1, dtype=torch.uint8, device=dev))
    assert e.value.code == 3
    assert ctypes.sizeof(dims) == 28


def test_requests_that_do_not_fit_are_reported(dev):
    import mla_decode_attention_06_gb300 as M
    c = Case("bf16", 15, **NARROW, qlens=(20, 30, 10), past=(0, 2000, 5))
    a, k = c.args(dev)
    k["total_keys"] = 300          # room for 2 + 3 tiles: the second request needs 16
    out = torch.zeros(c.T, c.H, c.V, dtype=torch.bfloat16, device=dev)
    with pytest.raises(M.MlaError) as e:
        M.mla_prefill_paged(*a, **k, out=out, debug=True)
    assert e.value.code == 5
    want, _ = c.expected()
    g = out.float().cpu().numpy()
    assert np.linalg.norm(g[:20] - want[:20]) <= TOL["f16"] * np.linalg.norm(want[:20])
    assert np.isnan(g[20:50]).all()


def test_bad_pages_are_dropped_and_reported(dev):
    import mla_decode_attention_06_gb300 as M
    c = Case("e2m1", 16, **NARROW, qlens=(40,), past=(100,))
    a, k = c.args(dev)
    a[3][0, 2] = c.num_pages + 5
    out = torch.zeros(c.T, c.H, c.V, dtype=torch.bfloat16, device=dev)
    with pytest.raises(M.MlaError) as e:
        M.mla_prefill_paged_fp4(*a, **k, out=out, debug=True)
    assert e.value.code == 5
    x = c.cached(0)
    keep = np.r_[0:32, 48:140]     # the keys of page 2 are gone, the others keep their positions
    want = np.zeros((c.T, c.H, c.V))
    for i in range(40):
        j = keep[keep <= 100 + i]
        s = c.scale * (np.einsum("hn,kl,hln->hk", ref.bf16_values(c.q)[i, :, :c.N], x[j, :c.L], c.uk) +
                       ref.bf16_values(c.q)[i, :, c.N:] @ x[j, c.L:].T)
        p = np.exp(s - s.max(1, keepdims=True))
        want[i] = np.einsum("hk,kl,hvl->hv", p / p.sum(1, keepdims=True), x[j, :c.L], c.uv)
    g = out.float().cpu().numpy()
    assert np.linalg.norm(g - want) <= TOL["f16"] * np.linalg.norm(want)


def test_matches_the_decode(dev):
    # the absorbed and the expanded form of the same call; the decode rounds four values to
    # bf16 (absorbed query with the softmax's factor of 2, P, latent output, output): 1.2e-2
    import mla_decode_attention_06_gb300 as M
    c = Case("e2m1", 17, **WIDE, H=16, ps=64, qlens=(3, 1, 2), past=(500, 90, 0))
    out, _ = call(c, dev)
    a, k = c.args(dev)
    k.pop("total_keys")
    want, _ = M.mla_decode_paged_fp4(*a, **k)
    d = (out.float() - want.float()).norm() / want.float().norm()
    assert d <= TOL["f16"] + 1.2e-2


def test_captured_and_replayed(dev):
    import mla_decode_attention_06_gb300 as M
    c = Case("bf16", 18, **WIDE, H=4, ps=64, qlens=(150, 20), past=(60, 300))
    d = Case("bf16", 19, **WIDE, H=4, ps=64, qlens=(150, 20), past=(60, 300), c=2.0 ** 20, q=2.0 ** -20)
    want_c, _ = call(c, dev)
    a, k = c.args(dev)
    out, ws = torch.empty_like(want_c), torch.empty(64 << 20, dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        M.mla_prefill_paged(*a, **k, out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want_c)
    # other inputs, among them ones that f16 does not hold: the sequence is chosen on the device
    for x, y in zip(a, d.args(dev)[0]):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    c.pool, c.table, c.q, c.uk, c.uv, c.rows = d.pool, d.table, d.q, d.uk, d.uv, d.rows
    want, _ = c.expected()
    assert np.linalg.norm(out.float().cpu().numpy() - want) <= TOL["bf16"] * np.linalg.norm(want)
    for x, y in zip(a, Case("bf16", 18, **WIDE, H=4, ps=64, qlens=(150, 20), past=(60, 300)).args(dev)[0]):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want_c)


@pytest.mark.parametrize("fmt", FORMATS)
def test_short_and_long_blocks_in_turn(dev, fmt):
    # many times more blocks than SMs, of one and of two sub-blocks, with and without keys: what one
    # of a block's roles skips must not let it run ahead into the next
    c = Case(fmt, 20, **NARROW, H=96, ps=16, qlens=(1, 300, 129, 0, 128, 500, 3, 260, 17, 400, 64, 5), past=(0, 0, 40, 9, 0, 0, 0, 0, 200, 0, -10, 0),
             pad=2)
    out, lse = call(c, dev, debug=False)
    compare(c, out, lse, "e4m3" if c.fmt == ref.E4M3 else "f16")
    first = out.clone()
    for _ in range(5):
        again, _ = call(c, dev, debug=False)
        assert torch.equal(again[:c.T], first[:c.T])


def test_short_and_long_blocks_in_turn_over_wide_heads(dev):
    c = Case("bf16", 21, **WIDE, H=64, ps=64, qlens=(1, 300, 129, 128, 420, 3, 260), past=(0,) * 7)
    check(c, dev)


def test_blocks_that_start_late_beside_others_that_raise_the_flag(dev):
    # one head past f16's range, most blocks of the expansion with a pair or two of their own, and
    # another stream's products on the SMs, so that blocks start while others end: all warps of a
    # block take the same decision, no wait runs out and the bits do not change
    c = Case("bf16", 22, **NARROW, H=96, qlens=(130, 70), past=(200, 0))
    c.w[1][40] = ref.bf16_bits(ref.bf16_values(c.w[1][40]) * 2.0 ** 30)
    c.uv = ref.bf16_values(c.w[1])
    first, lse = call(c, dev)
    compare(c, first, lse, "bf16")
    args = c.args(dev)
    x = torch.randn(2048, 2048, device=dev, dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s):
            for _ in range(4):
                torch.mm(x, x)
        out, _ = call(c, dev, args)
        assert torch.equal(out, first)


@pytest.mark.parametrize("small", [2.0 ** -13, 2.0 ** -22])
@pytest.mark.parametrize("fmt", FORMATS)
def test_small_rows_beside_large_ones(dev, fmt, small):
    # cached rows far smaller than their neighbours: a query that sees nothing else keeps its
    # relative precision (that of the bf16 sequence at least), token by token
    c = Case(fmt, 23, **WIDE, qlens=(150, 3), past=(0, 40))
    for b, keys in ((0, range(5)), (1, range(3, 31))):
        row = c.rows[b][list(keys)]
        if fmt == "bf16":
            v = ref.bf16_values(np.ascontiguousarray(c.pool[row, :2 * c.L]).view(np.uint16)) * small
            c.pool[row, :2 * c.L] = ref.bf16_bits(v).view(np.uint8)
        elif fmt == "e4m3":
            c.scales[row] *= np.float32(small)
        else:
            c.pool[row, c.L // 2:c.L // 2 + c.L // 32] -= np.uint8(-np.log2(small))
    out, lse = call(c, dev)
    want, want_lse = c.expected()
    g = out.float().cpu().numpy().astype(np.float64)
    kind = "bf16 e4m3" if fmt == "e4m3" else "bf16"
    for t in range(c.T):
        assert np.linalg.norm(g[t] - want[t]) <= TOL[kind] * np.linalg.norm(want[t]), t
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= TOL_LSE[kind]


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_weak_head_changes_no_other(dev, fmt):
    # one head's weights 2048 times smaller: the other heads' bits stay, its own values keep the
    # precision of the bf16 sequence at least
    kw = dict(**WIDE, H=3, qlens=(140, 9), past=(3, 150))
    want, want_lse = check(Case(fmt, 24, **kw), dev)
    c = Case(fmt, 24, **kw)
    for i, name in enumerate(("uk", "uv")):
        if fmt == "e4m3":
            c.w[i][1][1] *= np.float32(2.0 ** -11)
        else:
            c.w[i][1] = ref.bf16_bits(ref.bf16_values(c.w[i][1]) * 2.0 ** -11)
        getattr(c, name)[1] *= 2.0 ** -11
    out, lse = call(c, dev)
    for h in (0, 2):
        assert torch.equal(out[:, h], want[:, h]) and torch.equal(lse[:, h], want_lse[:, h])
    ref_out, ref_lse = c.expected()
    kind = "bf16 e4m3" if fmt == "e4m3" else "bf16"
    g = out[:, 1].float().cpu().numpy()
    assert np.linalg.norm(g - ref_out[:, 1]) <= TOL[kind] * np.linalg.norm(ref_out[:, 1])
    assert np.abs(lse[:, 1].cpu().numpy() - ref_lse[:, 1]).max() <= TOL_LSE[kind]


def test_widest_window(dev):
    # the largest window there is is no window, for query tokens before the first cached key too
    for past in ((40, 5), (-3, -100)):
        c = Case("bf16", 25, **NARROW, qlens=(20, 150), past=past, mask=2, window=2 ** 31 - 1)
        out, lse = call(c, dev, debug=past[0] >= 0)
        c.lens = c.lens.astype(np.int64)
        compare(c, out, lse, "f16")


@pytest.mark.parametrize("what", ["large", "small", "rope"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_request_out_of_range_changes_no_other(dev, fmt, what):
    # one request of a batch holds rows that f16 does not: the bits of the others are those of a batch
    # without it, over key splits and passes of heads too, and its own values are right
    import mla_decode_attention_06_gb300 as M
    scale = {"large": 2.0 ** -17, "small": None, "rope": 2.0 ** -23}[what]
    kw = dict(**NARROW, H=3, qlens=(140, 20, 300, 0, 5), past=(3, 250, 0, 40, 90), scale=scale, pad=2)
    clean, c = Case(fmt, 26, **kw), Case(fmt, 26, **kw)
    row = c.rows[1]
    if what == "rope":
        v = ref.bf16_values(np.ascontiguousarray(c.pool[row, -2 * c.R:]).view(np.uint16)) * 2.0 ** 20
        c.pool[row, -2 * c.R:] = ref.bf16_bits(v).view(np.uint8)
    else:
        k = 14 if what == "large" else -22
        if fmt == "bf16":
            v = ref.bf16_values(np.ascontiguousarray(c.pool[row, :2 * c.L]).view(np.uint16)) * 2.0 ** k
            c.pool[row, :2 * c.L] = ref.bf16_bits(v).view(np.uint8)
        elif fmt == "e4m3":
            c.scales[row] *= np.float32(2.0 ** k)
        else:
            at = c.pool[row, c.L // 2:c.L // 2 + c.L // 32].astype(np.int64) + k
            c.pool[row, c.L // 2:c.L // 2 + c.L // 32] = at.astype(np.uint8)
    others = np.r_[0:140, 160:465]
    want_all, want_lse_all = c.expected()
    for splits in (1, 3):
        want, want_lse = check(clean, dev, num_splits=splits)
        dims = M.MlaDims(num_heads=3, qk_nope=c.N, qk_rope=c.R, kv_lora_rank=c.L, v_head=c.V, page_size=c.ps, num_pages=c.num_pages)
        opts = M.MlaOpts(mask=1, window=0, scale=float(c.scale), num_splits=splits, flags=0)
        n = M.mla_prefill_workspace_size(dims, opts, c.fmt, 5, c.T + 2, int(c.lens.sum()))
        one_head = (int(c.lens.sum()) // 128 + 5) * 2 * 16384
        for heads in (3, 1):
            ws = torch.empty(n - (3 - heads) * one_head, dtype=torch.uint8, device=dev)
            out, lse = call(c, dev, num_splits=splits, workspace=ws)
            assert torch.equal(out[others], want[others]) and torch.equal(lse[others], want_lse[others])
            assert (out[c.T:] == 7).all() and (lse[c.T:] == 7).all()
            g, w = out[140:160].float().cpu().numpy().astype(np.float64), want_all[140:160]
            assert np.linalg.norm(g - w) <= TOL["bf16 e4m3" if fmt == "e4m3" else "bf16"] * np.linalg.norm(w)
            assert np.abs(lse[140:160].cpu().numpy() - want_lse_all[140:160]).max() <= TOL_LSE["bf16 e4m3" if fmt == "e4m3" else "bf16"]
