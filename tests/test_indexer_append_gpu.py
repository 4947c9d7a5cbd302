"""GPU: mla_indexer_append (index keys into the paged e4m3 cache, index queries as codes) against
plain 64-bit numpy forms, bit for bit: LayerNorm and rotation are each rounded once to bf16, codes
are those of exact quotients."""
import numpy as np
import pytest
import torch

import code_ref as cr
import latent_ref as ref

pytestmark = pytest.mark.gpu
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_decode_attention_06_gb300 import build
    build.build()
    return torch.device("cuda:0")


def bf16(bits, dev):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(dev).view(torch.bfloat16)


class Case(cr.Pages):
    def __init__(self, *, seed=1, D=128, H=3, R=64, ps=16, qlens=(1,), past=(0,), ln=True, weight=True, pad=0, wide=0):
        super().__init__(seed, ps, qlens, past)
        r, n = self.rng, self.T + pad
        self.D, self.H, self.R, self.n, self.wide = D, H, R, n, wide
        self.k = ref.bf16_bits(r.standard_normal((n, D)) * np.exp2(r.integers(-3, 4, (n, 1))) + 0.5)
        self.q = ref.bf16_bits(r.standard_normal((n, H, D)) * np.exp2(r.integers(-3, 4, (n, H, 1)))) if H else None
        self.weight = r.standard_normal((n, H)).astype(np.float32) if weight and H else None
        self.gamma = ref.bf16_bits(1 + 0.3 * r.standard_normal(D)) if ln else None
        self.beta = ref.bf16_bits(0.2 * r.standard_normal(D)) if ln else None
        self.freqs = None
        if R:
            ang = np.arange(max(1, int(self.lens.max())))[:, None] * 10000.0 ** (-2 * np.arange(R // 2) / R)
            self.freqs = ref.bf16_bits(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(len(ang), R))
        self.pool = r.integers(0, 256, (self.rows, D), np.uint8)
        self.scales = r.random(self.rows, np.float32)
        self.codes0 = r.integers(0, 256, (n, H, D), np.uint8)
        self.scales0 = r.random((n, H), np.float32)

    def expected(self):
        T, D, R = self.T, self.D, self.R
        live = np.flatnonzero((self.row >= 0) & (self.pos < (len(self.freqs) if R else 1 << 40)))
        k = self.k[:T]
        if self.gamma is not None:
            k = cr.layer_norm(k, self.gamma, self.beta, EPS)
        f = self.freqs[np.clip(self.pos, 0, len(self.freqs) - 1)] if R else None
        if R:
            k = np.concatenate([k[:, :D - R], cr.turn(k[:, D - R:], f)], 1)
        pool, scales = self.pool.copy(), self.scales.copy()
        codes, s = cr.encode(k, cr.E4M3)
        pool[self.row[live]], scales[self.row[live]] = codes[live], s[live]
        if not self.H:
            return pool, scales, None, None
        q = self.q[:T]
        if R:
            q = np.concatenate([q[..., :D - R], cr.turn(q[..., D - R:], f[:, None])], -1)
        codes, s = cr.encode(q.reshape(-1, D), cr.E4M3)
        s = s.reshape(T, self.H) * (self.weight[:T] if self.weight is not None else np.float32(1))
        q_codes, q_scales = self.codes0.copy(), self.scales0.copy()
        q_codes[live], q_scales[live] = codes.reshape(T, self.H, D)[live], s[live]
        return pool, scales, q_codes, q_scales

    def run(self, dev, debug=True, **kw):
        import mla_decode_attention_06_gb300 as M
        t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        b = lambda a: None if a is None else bf16(a, dev)  # noqa: E731
        k = torch.full((self.n, self.D + self.wide), float("nan"), dtype=torch.bfloat16, device=dev)
        k[:, :self.D] = bf16(self.k, dev)
        pool, scales = t(self.pool), t(self.scales)
        qc, qs = (t(self.codes0), t(self.scales0)) if self.H else (None, None)
        M.mla_indexer_append(k[:, :self.D], t(self.offsets), pool, scales, t(self.table), t(self.lens),
                             page_size=self.ps, freqs_cis=b(self.freqs), k_norm_gamma=b(self.gamma),
                             k_norm_beta=b(self.beta), epsilon=EPS, q=b(self.q), q_weight=t(self.weight), q_codes=qc,
                             q_scales=qs, debug=debug, **kw)
        torch.cuda.synchronize()
        return [None if x is None else x.cpu().numpy() for x in (pool, scales, qc, qs)]


def check(c, dev, **kw):
    for got, want in zip(c.run(dev, **kw), c.expected()):
        assert (got is None) == (want is None)
        if want is not None:
            assert np.array_equal(got, want, equal_nan=want.dtype == np.float32)


@pytest.mark.parametrize("D,R", [(128, 64), (128, 0), (64, 32), (64, 64), (8, 8), (96, 32), (40, 16), (256, 64), (136, 128)])
@pytest.mark.parametrize("ln", [True, False])
def test_widths_and_parts(dev, D, R, ln):
    check(Case(D=D, R=R, ln=ln, H=5, qlens=(5, 1, 0, 17), past=(9, 0, 3, 20), pad=2, wide=24), dev)


@pytest.mark.parametrize("H", [0, 1, 16, 63, 64, 65, 200])
def test_heads(dev, H):
    check(Case(H=H, qlens=(3, 30), past=(70, 0), weight=H != 16), dev)
    check(Case(H=H, D=64, R=0, qlens=(3, 30), past=(70, 0)), dev)


@pytest.mark.parametrize("H,D,R,tokens", [(64, 128, 64, 4870), (65, 128, 64, 2440), (4, 64, 64, 1003), (1, 128, 32, 100),
                                          (17, 96, 0, 333), (3, 8, 8, 70), (128, 64, 32, 50), (1, 16, 16, 1000)])
def test_tokens_of_a_block(dev, H, D, R, tokens):
    """One token after the other, and several side by side, in blocks that the last tokens leave part empty."""
    check(Case(D=D, R=R, H=H, qlens=(tokens - 37, 0, 30, 7), past=(0, 5, 11, 3), pad=3, ps=16), dev)


@pytest.mark.parametrize("B,ps", [(1, 1), (2, 8), (33, 24), (1100, 64)])
def test_many_requests_and_pages(dev, B, ps):
    r = np.random.default_rng(B)
    check(Case(seed=B, D=64, R=16, H=2, ps=ps, qlens=tuple(r.integers(0, 5, B - 1)) + (2,), past=tuple(r.integers(0, 40, B))), dev)


@pytest.mark.parametrize("ln", [True, False])
def test_values_at_the_edges(dev, ln):
    c = Case(D=128, R=64, H=12, qlens=(12,), ln=ln)
    v = c.rng.standard_normal((12, 128))
    v[0], v[1] = 0.0, 3.0
    v[2, 5], v[3, 100], v[4, 127] = np.nan, np.inf, -np.inf
    v[5] *= 2.0 ** 124
    v[6] *= 2.0 ** -130
    v[7, 64:] = 0.0
    v[8] = np.where(np.arange(128) % 2, 2.0 ** 100, -2.0 ** -100)
    v[9] = 448 * 2.0 ** -9
    v[10] = -0.0
    v[11] = 1000 + v[11] / 64
    c.k = ref.bf16_bits(v)
    c.q[3] = c.k
    check(c, dev)


def test_bad_pages_and_positions_are_skipped_and_reported(dev):
    import mla_decode_attention_06_gb300 as M
    c = Case(ps=8, D=64, R=32, H=4, qlens=(20, 30, 9, 4), past=(0, 5, 0, 0))
    c.table[0, 1] = -1
    c.table[1, 2] = c.num_pages
    c.lens[2] -= 4                      # four tokens before the start of the request
    c.pos[50:59] -= 4
    c.freqs = c.freqs[:30]              # request 1's last positions have no rotation
    c.lens[3] += 100
    c.pos[59:] += 100
    c.place()
    with pytest.raises(M.MlaError) as e:
        c.run(dev)
    assert e.value.code == 5
    check(c, dev, debug=False)


def test_the_indexer_reads_what_is_written(dev):
    """Append, then score: every key's score from the codes and scales written, exactly (whole numbers of
    2^-18 times powers of two, summed over few heads in fp64), in the indexer's order."""
    import mla_decode_attention_06_gb300 as M
    c = Case(D=128, R=64, H=4, ps=16, qlens=(50, 30), past=(0, 0))
    pool, scales, qc, qs = c.run(dev)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    rows, got = M.mla_indexer_fp8(t(qc), t(qs), t(c.offsets), t(pool), t(scales), t(c.table), t(c.lens), page_size=16,
                                  top_k=64, with_scores=True, debug=True)
    kv, qv = cr.E4M3_VALUES[pool], cr.E4M3_VALUES[qc]
    rows, got = rows.cpu().numpy(), got.cpu().numpy()
    for i in range(c.T):
        keys = c.row[(c.req == c.req[i]) & (c.pos <= c.pos[i])]
        s = np.zeros(len(keys))
        for h in range(c.H):
            s = s + (qs[i, h].astype(np.float64) * scales[keys].astype(np.float64)) * (kv[keys] @ qv[i, h])
        order = np.lexsort((np.arange(len(keys)), -s))
        n = min(64, len(keys))
        assert np.array_equal(rows[i, :n], keys[order][:n]) and (rows[i, n:] == -1).all()
        assert np.array_equal(got[i, :n], s[order][:n])


def test_streams_and_graph(dev):
    import mla_decode_attention_06_gb300 as M
    c = Case(qlens=(40,), past=(13,))
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    kw = dict(page_size=16, freqs_cis=bf16(c.freqs, dev), k_norm_gamma=bf16(c.gamma, dev), k_norm_beta=bf16(c.beta, dev),
              epsilon=EPS, q=bf16(c.q, dev), q_weight=t(c.weight))
    pools = [(t(c.pool), t(c.scales)) for _ in range(2)]
    head, tail = (bf16(c.k, dev), t(c.offsets)), (t(c.table), t(c.lens))
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    a = M.mla_indexer_append(*head, *pools[0], *tail, **kw, stream=side)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = M.mla_indexer_append(*head, *pools[1], *tail, **kw)
    graph.replay()
    want = c.expected()
    for got in ((*pools[0], *a), (*pools[1], *b)):
        for x, y in zip(got, want):
            assert np.array_equal(x.view(torch.uint8).cpu().numpy(), np.ascontiguousarray(y).view(np.uint8))


def test_offsets_past_32_bits(dev):
    """The last pages of an index cache of more than 2^32 bytes."""
    import mla_decode_attention_06_gb300 as M
    c = Case(qlens=(100, 30), past=(0, 40), ps=64, H=2)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    base = (1 << 32) // (64 * 128) + 5
    pool = torch.empty((base + c.num_pages) * 64, 128, dtype=torch.uint8, device=dev)
    scales = torch.empty(len(pool), device=dev)
    pool[base * 64:], scales[base * 64:] = t(c.pool), t(c.scales)
    table = np.where(c.table >= 0, c.table + base, -1).astype(np.int32)
    M.mla_indexer_append(bf16(c.k, dev), t(c.offsets), pool, scales, t(table), t(c.lens), page_size=64,
                         freqs_cis=bf16(c.freqs, dev), k_norm_gamma=bf16(c.gamma, dev), k_norm_beta=bf16(c.beta, dev),
                         epsilon=EPS, debug=True)
    want = c.expected()
    assert np.array_equal(pool[base * 64:].cpu().numpy(), want[0])
    assert np.array_equal(scales[base * 64:].cpu().numpy(), want[1])
