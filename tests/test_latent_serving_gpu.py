"""GPU: the latent-cache operators as a server runs them: prompts appended and attended, then one
token at a time appended and decoded (captured once, replayed), over every cache format; calls
side by side, graphs that share a workspace, pools past 32-bit offsets.

The appended rows are compared bit for bit.  Tolerances of the outputs, relative 2-norms against
64-bit arithmetic on the rows that the cache holds, one bf16 rounding being 2.3e-3 rms at worst and
the softmax doubling the error of a score: prefill as in its own tests (3.5e-3; e4m3 5.1e-3); the
bf16 decode rounds the absorbed query (factor 2), P, the latent output and the output:
2.3e-3 * sqrt(4 + 3) = 6.1e-3; the e4m3 decode also w_uk and the rows as keys (factor 2 each), the
rows as values and w_uv: 2.3e-3 * sqrt(7 + 8 + 2) = 9.5e-3; the e2m1 decode 4.0e-3 (f16 operands).
"""
import numpy as np
import pytest
import torch

import latent_ref as ref

pytestmark = pytest.mark.gpu

FORMATS = {"bf16": ref.BF16, "e4m3": ref.E4M3, "e2m1": ref.E2M1}
TOL_PREFILL = {"bf16": 3.5e-3, "e4m3": 5.1e-3, "e2m1": 3.5e-3}
TOL_DECODE = {"bf16": 6.1e-3, "e4m3": 9.5e-3, "e2m1": 4.0e-3}
N, R, L, V, H, PS, EPS = 128, 64, 512, 128, 16, 64, 1e-6


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


class Server:
    """Requests over one pool, with the 64-bit reference beside it."""

    def __init__(self, fmt, dev, seed, B, max_len, base_page=0):
        import mla_decode_attention_06_gb300 as M
        self.M, self.fmt, self.dev, self.B = M, fmt, dev, B
        self.r = r = np.random.default_rng(seed)
        self.code = FORMATS[fmt]
        per = -(-max_len // PS)
        self.num_pages = base_page + B * per + 1
        self.table = base_page + r.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
        width = M.mla_cache_row_bytes(self.code, L, R)
        self.pool = torch.empty(self.num_pages, PS, width, dtype=torch.uint8, device=dev)
        self.pool[base_page:] = 0xFF
        self.scales = torch.full((self.num_pages * PS,), float("nan"), device=dev) if fmt == "e4m3" else None
        self.freqs = ref.bf16_bits(r.standard_normal((max_len, R)))
        self.gamma = ref.bf16_bits(r.random(L) + 0.5)
        uk, uv = r.standard_normal((H, L, N)) / np.sqrt(N), r.standard_normal((H, V, L)) / np.sqrt(L)
        if fmt == "e4m3":
            self.w, self.uk, self.uv = [], None, None
            for name, w in (("uk", uk), ("uv", uv)):
                s = (np.abs(w).max() / 448 * (1 + r.random((H, -(-w.shape[1] // 128), -(-w.shape[2] // 128))))).astype(np.float32)
                full = s.repeat(128, 1)[:, :w.shape[1]].repeat(128, 2)[:, :, :w.shape[2]].astype(np.float64)
                code = ref.nearest_code(np.abs(w) / full, ref.e4m3_grid()).astype(np.uint8)
                setattr(self, name, ref.e4m3_grid()[code] * np.where(w < 0, -1.0, 1.0) * full)
                self.w += [torch.from_numpy(code | (w < 0).astype(np.uint8) << 7).to(dev), torch.from_numpy(s).to(dev)]
        else:
            b = [ref.bf16_bits(uk), ref.bf16_bits(uv)]
            self.uk, self.uv = (ref.bf16_values(x) for x in b)
            self.w = [bf16(x, dev) for x in b]
        self.t_table, self.t_freqs, self.t_gamma = (torch.from_numpy(self.table).to(dev), bf16(self.freqs, dev),
                                                    bf16(self.gamma, dev))
        self.cached = [np.zeros((0, L + R)) for _ in range(B)]     # the values that the rows stand for
        self.bytes = [np.zeros((0, width), np.uint8) for _ in range(B)]

    def tokens(self, qlens, pad=0):
        """New tokens: bits of their rows in a wider buffer, their queries, offsets."""
        T = int(sum(qlens)) + pad
        new = ref.bf16_bits(self.r.standard_normal((T, L + R + 192)))
        q = ref.bf16_bits(self.r.standard_normal((T, H, N + R)))
        return new, q, np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)

    def expect(self, new, q, offsets):
        """Appends to the reference cache; returns the turned queries' bits and the outputs."""
        T = int(offsets[-1])
        lens = np.array([len(c) for c in self.cached]) + np.diff(offsets)
        pos = np.concatenate([np.arange(l - n, l) for l, n in zip(lens, np.diff(offsets))]).astype(int)
        y, rope, q2 = ref.append(new[:T, 192:], self.gamma, self.freqs, pos, EPS, L, R, q[:T], N)
        rows, scales = ref.encode(y, rope, self.code)
        values = ref.decode(rows, scales, self.code, L, R)
        for b in range(self.B):
            s = slice(offsets[b], offsets[b + 1])
            self.cached[b] = np.concatenate([self.cached[b], values[s]])
            self.bytes[b] = np.concatenate([self.bytes[b], rows[s]])
        out, _ = ref.attention(ref.bf16_values(q2), self.uk, self.uv, self.cached, lens, offsets, 1 / np.sqrt(N + R), 1, 0)
        return q2, out

    def append(self, new, q, offsets, lens, **kw):
        self.M.mla_cache_append(new, offsets, self.pool, self.t_table, lens, self.t_freqs, self.t_gamma, page_size=PS,
                                epsilon=EPS, cache_format=self.code, kv_scales=self.scales, q=q, **kw)

    def attend(self, kind, q, offsets, lens, **kw):
        M, cache = self.M, [self.pool] + ([self.scales] if self.fmt == "e4m3" else [])
        if self.fmt == "bf16":
            cache = [self.pool.view(torch.bfloat16)]
        fn = {"prefill": (M.mla_prefill_paged, M.mla_prefill_paged_fp8, M.mla_prefill_paged_fp4),
              "decode": (M.mla_decode_paged, M.mla_decode_paged_fp8, M.mla_decode_paged_fp4)}[kind][self.code]
        return fn(q, offsets, *cache, self.t_table, lens, *self.w, page_size=PS, **kw)[0]

    def check_cache(self):
        rows = self.pool.cpu().numpy().reshape(-1, self.pool.shape[2])
        for b, want in enumerate(self.bytes):
            j = np.arange(len(want))
            assert np.array_equal(rows[self.table[b, j // PS].astype(np.int64) * PS + j % PS], want)


def close(got, want, tol):
    g = got.float().cpu().numpy().astype(np.float64)[:len(want)]
    err = np.linalg.norm(g - want) / np.linalg.norm(want)
    assert err <= tol, err


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("prompts", [(90, 1, 200), (1,)])
def test_prompts_then_tokens(dev, fmt, prompts):
    B, pad = len(prompts), 3
    s = Server(fmt, dev, 31, B, max(prompts) + 4)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    new, q, offsets = s.tokens(prompts, pad)
    d_new, d_q, d_off, d_lens = bf16(new, dev), bf16(q, dev), t(offsets), t(np.array(prompts, np.int32))
    s.append(d_new[:, 192:], d_q, d_off, d_lens, debug=True)                 # rows of a wider projection, q in place
    out = torch.full((len(q), H, V), 7.0, dtype=torch.bfloat16, device=dev)
    s.attend("prefill", d_q, d_off, d_lens, total_keys=sum(prompts), out=out, debug=True)
    q2, want = s.expect(new, q, offsets)
    s.check_cache()
    assert np.array_equal(bits(d_q)[:len(q2)], q2) and np.array_equal(bits(d_q)[len(q2):], q[len(q2):])
    close(out, want, TOL_PREFILL[fmt])
    assert (out[len(want):] == 7).all()

    # one token a request: the step is captured once and replayed, its inputs copied in
    d_off = t(np.arange(B + 1, dtype=np.int32))
    d_new, d_q = d_new[:B].clone(), d_q[:B].clone()
    d_lens = t(np.ones(B, np.int32))                                           # any valid value while capturing
    ws, side, g = torch.empty(64 << 20, dtype=torch.uint8, device=dev), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.append(d_new[:, 192:], d_q, d_off, d_lens)
        out = s.attend("decode", d_q, d_off, d_lens, workspace=ws)
    for step in range(3):
        new, q, offsets = s.tokens([1] * B)
        d_new.copy_(bf16(new, dev))
        d_q.copy_(bf16(q, dev))
        d_lens.copy_(t(np.array(prompts, np.int32) + step + 1))
        g.replay()
        q2, want = s.expect(new, q, offsets)
        s.check_cache()
        assert np.array_equal(bits(d_q), q2)
        close(out, want, TOL_DECODE[fmt])


def filled(fmt, dev, seed, lens, base_page=0):
    s = Server(fmt, dev, seed, len(lens), max(lens), base_page)
    new, q, offsets = s.tokens(lens)
    args = bf16(q, dev), torch.from_numpy(offsets).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
    s.append(bf16(new, dev)[:, 192:], *args, debug=True)
    last = args[0][torch.from_numpy(offsets[1:].astype(np.int64) - 1).to(dev)].contiguous()
    one = torch.arange(len(lens) + 1, dtype=torch.int32, device=dev)
    return s, args, (last, one, args[2])


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_offsets_past_32_bits(dev, fmt):
    # the same pages at the start of a pool and behind 4 GiB of it: the same bits
    lens = (300, 70)
    outs = []
    for base in (0, (1 << 32) // (PS * {"bf16": 1152, "e4m3": 640, "e2m1": 400}[fmt]) + 1):
        s, prompt, one = filled(fmt, dev, 32, lens, base)
        outs.append((s.attend("prefill", *prompt, total_keys=sum(lens), debug=True), s.attend("decode", *one, debug=True),
                     s.pool[base:].clone()))
        del s
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_graphs_that_share_a_workspace(dev):
    big, _, one = filled("e2m1", dev, 33, (900, 64, 1, 333))
    small, prompt, _ = filled("e2m1", dev, 34, (140,))
    want = [big.attend("decode", *one), small.attend("prefill", *prompt, total_keys=140),
            big.attend("decode", *one, num_splits=7)]
    ws, side, graphs, outs = torch.empty(64 << 20, dtype=torch.uint8, device=dev), torch.cuda.Stream(), [], []
    for call in (lambda: big.attend("decode", *one, workspace=ws),
                 lambda: small.attend("prefill", *prompt, total_keys=140, workspace=ws),
                 lambda: big.attend("decode", *one, num_splits=7, workspace=ws)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(call())
    for i in (0, 1, 2, 1, 0, 0, 2, 2, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want[i])


def test_calls_side_by_side(dev):
    # two streams, no workspace given: each call has its own
    a, _, one = filled("e2m1", dev, 35, (2000, 64, 1, 333))
    b, prompt, _ = filled("bf16", dev, 36, (700, 20))
    want = a.attend("decode", *one), b.attend("prefill", *prompt, total_keys=720)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((a.attend("decode", *one, stream=s1), b.attend("prefill", *prompt, total_keys=720, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("op", ["prefill", "decode e2m1", "decode bf16", "decode sparse", "indexer"])
def test_a_stream_of_its_own_leaves_freed_memory_alone(dev, op):
    # memory that the current stream has given back but still reads, of the sizes that the call
    # asks for: a call on another stream must not write there
    import mla_decode_attention_06_gb300 as M
    r = np.random.default_rng(50)
    T, rows = 24, 24 * 128
    t = lambda a, d=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(dev, d)  # noqa: E731
    offsets, table, lens = t(np.arange(T + 1)), t(np.arange(2 * T).reshape(T, 2)), t(np.full(T, 100))
    rand = lambda *shape: t(r.standard_normal(shape), torch.bfloat16)  # noqa: E731
    q, uk, uv = rand(T, H, N + R), rand(H, L, N) / N ** 0.5, rand(H, V, L) / L ** 0.5
    pool = rand(rows, L + R)
    dims = M.MlaDims(num_heads=H, qk_nope=N, qk_rope=R, kv_lora_rank=L, v_head=V, page_size=PS, num_pages=2 * T)
    opts = M.MlaOpts(mask=1, window=0, scale=0.07, num_splits=0, flags=0)
    size = M.mla_decode_workspace_size(dims, opts, T, T)
    kw = dict(page_size=PS, scale=0.07)
    if op == "prefill":
        size = M.mla_prefill_workspace_size(dims, opts, 0, T, T, 100 * T)
        call = lambda **k: M.mla_prefill_paged(q, offsets, pool, table, lens, uk, uv, total_keys=100 * T, **kw, **k)[0]  # noqa: E731
    elif op == "decode e2m1":
        pool4 = t(r.integers(0, 120, (rows, 400)), torch.uint8)
        call = lambda **k: M.mla_decode_paged_fp4(q, offsets, pool4, table, lens, uk, uv, **kw, **k)[0]  # noqa: E731
        pool4[:, 256:272] = 127
        pool4[:, 272:] = pool.view(torch.uint8)[:, 2 * L:]
    elif op == "decode bf16":
        call = lambda **k: M.mla_decode_paged(q, offsets, pool, table, lens, uk, uv, **kw, **k)[0]  # noqa: E731
    elif op == "decode sparse":
        rows_of = t(r.integers(0, rows, (T, 64)))
        call = lambda **k: M.mla_decode_sparse(q, offsets, pool, rows_of, None, uk, uv, **kw, **k)[0]  # noqa: E731
    else:
        codes = [t(r.integers(0, 120, s), torch.uint8) for s in ((T, 4, 64), (rows, 64))]
        ones = [torch.ones(T, 4, device=dev), torch.ones(rows, device=dev)]
        size = 0
        call = lambda **k: M.mla_indexer_fp8(codes[0], ones[0], offsets, codes[1], ones[1], table, lens, page_size=PS,  # noqa: E731
                                             top_k=32, **k)[0]
    want = call().clone()
    s = torch.cuda.Stream()
    call(stream=s)                       # one-time set-up of the call
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full_like(want, 3), torch.full((max(size, 1),), 7, dtype=torch.uint8, device=dev)]
    seen = [torch.empty_like(x) for x in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)       # about 0.2 s
    for a, b in zip(seen, held):
        a.copy_(b)
    del a, b, held
    got = call(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert (seen[0] == 3).all() and (seen[1] == 7).all()
