"""GPU: mla_cache_read (rows of the paged latent cache as bf16 values) against plain 64-bit numpy,
bit for bit: each value is one rounding of a code times its scale."""
import numpy as np
import pytest
import torch

import code_ref as cr
import latent_ref as ref

pytestmark = pytest.mark.gpu
FORMATS = {"bf16": ref.BF16, "e4m3": ref.E4M3, "e2m1": ref.E2M1}
WIDTHS = {"wide": (512, 64), "narrow": (64, 16), "odd": (96, 40), "widest": (512, 128)}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_decode_attention_06_gb300 import build
    build.build()
    return torch.device("cuda:0")


def same(a, b):
    nan = (a & 0x7FFF) > 0x7F80
    return np.array_equal(nan, (b & 0x7FFF) > 0x7F80) and np.array_equal(a[~nan], b[~nan])


class Case(cr.Pages):
    def __init__(self, fmt, L, R, *, seed=1, ps=16, qlens=(1,), past=(0,)):
        super().__init__(seed, ps, qlens, past)
        r, n = self.rng, self.rows
        self.fmt, self.L, self.R = fmt, L, R
        y = ref.bf16_bits(r.standard_normal((n, L)) * np.exp2(r.integers(-3, 4, (n, 1))))
        self.pool, _ = ref.encode(y, ref.bf16_bits(r.standard_normal((n, R))), fmt)
        self.scales = None
        if fmt == ref.E4M3:     # any scale, codes of every value among them NaN
            self.scales = np.exp(2 * r.standard_normal(n)).astype(np.float32)
            self.pool[::5, :L] = r.integers(0, 256, (len(self.pool[::5]), L))

    def expected(self):
        rows = ref.decode(self.pool, self.scales, self.fmt, self.L, self.R)
        with np.errstate(all="ignore"):
            return np.where(self.row[:, None] >= 0, ref.bf16_bits(rows[self.row]), 0x7FC0)

    def read(self, dev, pad=0, debug=True, **kw):
        import mla_decode_attention_06_gb300 as M
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        out = torch.full((self.T + pad, self.L + self.R), float("nan"), dtype=torch.bfloat16, device=dev)
        got = M.mla_cache_read(t(self.offsets), t(self.pool), t(self.table), t(self.lens), kv_lora_rank=self.L,
                               qk_rope=self.R, page_size=self.ps, cache_format=self.fmt,
                               kv_scales=None if self.scales is None else t(self.scales), out=out, debug=debug, **kw)
        torch.cuda.synchronize()
        assert got is out
        return out.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("ps", [1, 8, 16, 24, 64])
def test_formats_widths_pages(dev, fmt, width, ps):
    c = Case(FORMATS[fmt], *WIDTHS[width], ps=ps, qlens=(5, 1, 0, 70, 33), past=(9, 0, 3, 20, 0))
    got = c.read(dev, pad=3)
    assert same(got[:c.T], c.expected())
    assert ((got[c.T:] & 0x7FFF) > 0x7F80).all()      # rows behind the last request keep what they held


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [1, 2, 31, 33, 1200])
def test_many_requests(dev, fmt, B):
    r = np.random.default_rng(B)
    c = Case(FORMATS[fmt], 64, 16, seed=B, ps=8, qlens=tuple(r.integers(0, 9, B - 1)) + (3,), past=tuple(r.integers(0, 9, B)))
    assert same(c.read(dev), c.expected())


def test_codes_at_the_edges(dev):
    """Every e2m1 code under every scale (255 is NaN), every e4m3 code under scales at fp32's ends."""
    L, R = 64, 16
    c = Case(ref.E2M1, L, R, ps=64, qlens=(256,))
    c.pool[:, :L // 2] = np.arange(16)[:, None].repeat(2, 0).reshape(1, -1) * 17
    c.pool[c.row, L // 2] = np.arange(256)
    c.pool[c.row, L // 2 + 1] = np.arange(256)[::-1]
    assert same(c.read(dev), c.expected())
    c = Case(ref.E4M3, 256, R, ps=64, qlens=(40,))
    c.pool[:, :256] = np.arange(256)
    c.scales[c.row] = np.concatenate([np.float32([0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 3e38, np.inf, np.nan, 2.0 ** -133,
                                                  1 + 2.0 ** -23, 1 - 2.0 ** -24]),
                                      np.random.default_rng(2).integers(0, 1 << 31, 30).astype(np.uint32).view(np.float32)])
    with np.errstate(all="ignore"):
        assert same(c.read(dev), c.expected())


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_pages_and_positions_are_left_and_reported(dev, fmt):
    import mla_decode_attention_06_gb300 as M
    c = Case(FORMATS[fmt], 64, 16, ps=8, qlens=(20, 30, 9, 4), past=(0, 5, 0, 0))
    c.table[0, 1] = -1
    c.table[1, 2] = c.num_pages
    c.lens[2] -= 4                      # four tokens before the start of the request
    c.pos[50:59] -= 4
    c.lens[3] += 100                    # past the block table
    c.pos[59:] += 100
    c.place()
    assert (c.row < 0).sum() == 8 + 8 + 4 + 4
    with pytest.raises(M.MlaError) as e:
        c.read(dev)
    assert e.value.code == 5
    got = c.read(dev, debug=False)
    assert same(got, c.expected())


def test_refusals_streams_and_graph(dev):
    import mla_decode_attention_06_gb300 as M
    c = Case(ref.E2M1, 512, 64, qlens=(100,), past=(13,))
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    args = (t(c.offsets), t(c.pool), t(c.table), t(c.lens))
    kw = dict(kv_lora_rank=512, qk_rope=64, page_size=16, cache_format=ref.E2M1)
    with pytest.raises(ValueError):
        M.mla_cache_read(*args, **kw)
    with pytest.raises(ValueError):
        M.mla_cache_read(*args, **kw, out=torch.empty(100, 512, dtype=torch.bfloat16, device=dev))
    with pytest.raises(M.MlaError):
        M.mla_cache_read(*args, **kw, total_rows=100, kv_scales=torch.ones(c.rows, device=dev))
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    a = M.mla_cache_read(*args, **kw, total_rows=100, stream=side)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = M.mla_cache_read(*args, **kw, total_rows=100)
    graph.replay()
    for x in (a, b):
        assert same(x.view(torch.int16).cpu().numpy().view(np.uint16), c.expected())
    assert M.mla_cache_read(t(np.zeros(2, np.int32)), *args[1:], **kw, total_rows=0).shape == (0, 576)


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_past_32_bits(dev, fmt):
    """The last pages of a pool of more than 2^32 bytes."""
    import mla_decode_attention_06_gb300 as M
    c = Case(FORMATS[fmt], 512, 64, ps=64, qlens=(100, 30), past=(0, 40))
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    base = (1 << 32) // (64 * c.pool.shape[1]) + 5
    pool = torch.empty((base + c.num_pages) * 64, c.pool.shape[1], dtype=torch.uint8, device=dev)
    pool[base * 64:] = t(c.pool)
    scales = None
    if c.scales is not None:
        scales = torch.empty(len(pool), device=dev)
        scales[base * 64:] = t(c.scales)
    table = np.where(c.table >= 0, c.table + base, -1).astype(np.int32)
    got = M.mla_cache_read(t(c.offsets), pool, t(table), t(c.lens), kv_lora_rank=512, qk_rope=64, page_size=64,
                           total_rows=c.T, cache_format=FORMATS[fmt], kv_scales=scales, debug=True)
    assert same(got.view(torch.int16).cpu().numpy().view(np.uint16), c.expected())
