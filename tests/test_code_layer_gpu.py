"""GPU: the operators over 8-bit codes as a sparse attention layer runs them.

  h += x, norm, codes -> down projection -> latents (norm, codes -> queries, index queries), cache rows, index
  keys -> append, index append -> prefill (prompts) or indexer, sparse decode (a token a request)
  -> codes -> output projection -> the next layer's x

for prompts and then token by token, the token step captured once and replayed.  Every stage is compared
with a plain form of what it was given: bit for bit where the operator's results are roundings of exact
values, the projections within K / 16 * 2^-22 of the sum of magnitudes and half a bf16 step (2^-8), the
attention within a relative 2-norm of 6.1e-3 (decode: the bf16 roundings of the absorbed query, which
counts twice, of P, the latent output and the output, each 2.3e-3 rms at worst: 2.3e-3 * sqrt(7)) and
3.5e-3 (prefill, f16 operands)."""
import numpy as np
import pytest
import torch

import code_ref as cr
import latent_ref as ref

pytestmark = pytest.mark.gpu
D, QR, H, N, R, L, V, HI, DI, PS, EPS, TOP = 512, 256, 4, 32, 32, 64, 32, 4, 64, 16, float(np.float32(1e-6)), 24
KINDS = {"int8": cr.INT8, "fp8": cr.E4M3}


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


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


class Layer:
    def __init__(self, kind, dev, seed, B, max_len):
        import mla_decode_attention_06_gb300 as M
        self.M, self.kind, self.fmt, self.dev, self.B = M, kind, KINDS[kind], dev, B
        r = self.r = np.random.default_rng(seed)
        self.linear = M.mla_linear_int8 if kind == "int8" else M.mla_linear_fp8
        per = -(-max_len // PS)
        self.table = r.permutation(B * per + 1)[:B * per].reshape(B, per).astype(np.int32)
        pages = B * per + 1
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.t = t
        self.t_table = t(self.table)
        self.pool = torch.full((pages, PS, L + R), float("nan"), dtype=torch.bfloat16, device=dev)
        self.k_cache = torch.full((pages * PS, DI), 0x7F, dtype=torch.uint8, device=dev)
        self.k_scales = torch.full((pages * PS,), float("nan"), device=dev)
        self.freqs = ref.bf16_bits(np.stack([np.cos(r.random((max_len, R // 2)) * 6), np.sin(r.random((max_len, R // 2)) * 6)],
                                            -1).reshape(max_len, R))
        vec = lambda n, s=0.3, m=1: ref.bf16_bits(m + s * r.standard_normal(n))  # noqa: E731
        self.g1, self.g2, self.gkv, self.gi, self.bi = vec(D), vec(QR), vec(L), vec(DI), vec(DI, 0.2, 0)
        self.tg = {k: bf16(getattr(self, k), dev) for k in ("g1", "g2", "gkv", "gi", "bi", "freqs")}
        self.w = {}
        for name, n, k in (("down", QR + L + R + DI, D), ("q", H * (N + R), QR), ("qi", HI * DI, QR), ("o", D, H * V)):
            c, s = cr.encode(ref.bf16_bits(r.standard_normal((n, k)) / np.sqrt(k)), self.fmt)
            self.w[name] = (t(c).view(torch.int8 if kind == "int8" else torch.float8_e4m3fn), t(s))
        self.uk, self.uv = ref.bf16_bits(r.standard_normal((H, L, N)) / np.sqrt(N)), ref.bf16_bits(r.standard_normal((H, V, L)) / 8)
        self.weight = r.random(HI).astype(np.float32) + 0.5
        self.t_w = (bf16(self.uk, dev), bf16(self.uv, dev))

    def step(self, x, h, offsets, lens, total=None):
        """One pass; h is updated in place.  Returns what the stages made."""
        M, T = self.M, x.shape[0]
        c1, s1, _ = M.mla_rmsnorm_quant(x, self.tg["g1"], epsilon=EPS, code_format=self.fmt, residual=h)
        down = self.linear(c1, s1, *self.w["down"])
        c2, s2, _ = M.mla_rmsnorm_quant(down[:, :QR], self.tg["g2"], epsilon=EPS, code_format=self.fmt)
        q = self.linear(c2, s2, *self.w["q"])
        qi = self.linear(c2, s2, *self.w["qi"])
        q_out = torch.empty_like(q)
        M.mla_cache_append(down[:, QR:QR + L + R], offsets, self.pool, self.t_table, lens, self.tg["freqs"], self.tg["gkv"],
                           page_size=PS, epsilon=EPS, q=q.view(T, H, N + R), q_out=q_out.view(T, H, N + R))
        weight = self.t(self.weight).expand(T, HI).contiguous() if not torch.cuda.is_current_stream_capturing() else self.step_weight
        qc, qs = M.mla_indexer_append(down[:, QR + L + R:], offsets, self.k_cache, self.k_scales, self.t_table, lens,
                                      page_size=PS, freqs_cis=self.tg["freqs"], k_norm_gamma=self.tg["gi"],
                                      k_norm_beta=self.tg["bi"], epsilon=EPS, q=qi.view(T, HI, DI), q_weight=weight)
        rows = None
        if total is None:
            rows, _ = M.mla_indexer_fp8(qc, qs, offsets, self.k_cache, self.k_scales, self.t_table, lens, page_size=PS, top_k=TOP)
            o, _ = M.mla_decode_sparse(q_out.view(T, H, N + R), offsets, self.pool, rows, None, *self.t_w, page_size=PS)
        else:
            o, _ = M.mla_prefill_paged(q_out.view(T, H, N + R), offsets, self.pool, self.t_table, lens, *self.t_w, page_size=PS,
                                       total_keys=total)
        c3, s3, _ = M.mla_rmsnorm_quant(o.view(T, H * V), code_format=self.fmt)
        y = self.linear(c3, s3, *self.w["o"])
        return dict(c1=c1, s1=s1, down=down, c2=c2, s2=s2, q=q, qi=qi, q_out=q_out, qc=qc, qs=qs, rows=rows, o=o, c3=c3, s3=s3, y=y)

    # ---------------------------------------------------------------- checks

    def check_codes(self, codes, scales, y):
        c, s = cr.encode(y, self.fmt)
        assert np.array_equal(raw(codes), c) and np.array_equal(scales.cpu().numpy(), s)

    def check_linear(self, out, codes, scales, w):
        x, xs, wc, ws = codes.double(), scales.double()[:, None], w[0].double(), w[1].double()
        want, room = (x @ wc.T) * xs * ws, (x.abs() @ wc.abs().T) * xs * ws * (-(-x.shape[1] // 16) * 2.0 ** -22)
        assert ((out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -22) + room).all()

    def check(self, got, x, h_before, h, offsets, lens):
        T, g = int(offsets[-1]), {k: None if v is None else v for k, v in got.items()}
        hb, y = cr.rmsnorm(bits(x), bits(h_before), self.g1, EPS)
        assert np.array_equal(bits(h), hb)
        self.check_codes(g["c1"], g["s1"], y)
        self.check_linear(g["down"], g["c1"], g["s1"], self.w["down"])
        down = bits(g["down"])
        self.check_codes(g["c2"], g["s2"], cr.rmsnorm(down[:, :QR], None, self.g2, EPS)[1])
        self.check_linear(g["q"], g["c2"], g["s2"], self.w["q"])
        self.check_linear(g["qi"], g["c2"], g["s2"], self.w["qi"])
        pos = np.concatenate([np.arange(l - n, l) for l, n in zip(lens, np.diff(offsets))]).astype(np.int64)
        req = np.repeat(np.arange(self.B), np.diff(offsets))
        row = self.table[req, pos // PS].astype(np.int64) * PS + pos % PS
        c, rope, q2 = ref.append(down[:, QR:QR + L + R], self.gkv, self.freqs, pos, EPS, L, R, bits(g["q"]).reshape(T, H, N + R), N)
        assert np.array_equal(bits(g["q_out"]).reshape(T, H, N + R), q2)
        assert np.array_equal(bits(self.pool).reshape(-1, L + R)[row], np.concatenate([c, rope], 1))
        k = cr.layer_norm(down[:, QR + L + R:], self.gi, self.bi, EPS)
        k = np.concatenate([k[:, :DI - R], cr.turn(k[:, DI - R:], self.freqs[pos])], 1)
        kc, ks = cr.encode(k, cr.E4M3)
        assert np.array_equal(raw(self.k_cache)[row], kc) and np.array_equal(self.k_scales.cpu().numpy()[row], ks)
        qi = bits(g["qi"]).reshape(T, HI, DI)
        qi = np.concatenate([qi[..., :DI - R], cr.turn(qi[..., DI - R:], self.freqs[pos][:, None])], -1)
        qc, qs = cr.encode(qi.reshape(-1, DI), cr.E4M3)
        assert np.array_equal(raw(g["qc"]).reshape(-1, DI), qc)
        assert np.array_equal(g["qs"].cpu().numpy(), qs.reshape(T, HI) * self.weight)
        # attention over the rows that the cache holds, or that the index scores choose
        cached = ref.bf16_values(bits(self.pool)).reshape(-1, L + R)
        place = [self.table[b, np.arange(n) // PS].astype(np.int64) * PS + np.arange(n) % PS for b, n in enumerate(lens)]
        if g["rows"] is None:
            want, _ = ref.attention(ref.bf16_values(q2), ref.bf16_values(self.uk), ref.bf16_values(self.uv),
                                    [cached[p] for p in place], lens, offsets, 1 / np.sqrt(N + R), 1, 0)
            tol = 3.5e-3
        else:
            kv, qv = cr.E4M3_VALUES[raw(self.k_cache)], cr.E4M3_VALUES[raw(g["qc"])]
            ksc, qsc = self.k_scales.cpu().numpy().astype(np.float64), g["qs"].cpu().numpy().astype(np.float64)
            chosen = []
            for b, p in enumerate(place):
                s = np.zeros(len(p))
                for i in range(HI):
                    s = s + (qsc[b, i] * ksc[p]) * (kv[p] @ qv[b, i])
                best = p[np.lexsort((np.arange(len(p)), -s))][:TOP]
                assert np.array_equal(g["rows"][b].cpu().numpy()[:len(best)], best)
                chosen.append(best)
            n = [len(c) for c in chosen]
            want, _ = ref.attention(ref.bf16_values(q2), ref.bf16_values(self.uk), ref.bf16_values(self.uv),
                                    [cached[c] for c in chosen], n, offsets, 1 / np.sqrt(N + R), 0, 0)
            tol = 6.1e-3
        o = g["o"].double().cpu().numpy()
        assert np.linalg.norm(o - want) <= tol * np.linalg.norm(want)
        self.check_codes(g["c3"], g["s3"], bits(g["o"]).reshape(T, H * V))
        self.check_linear(g["y"], g["c3"], g["s3"], self.w["o"])


@pytest.mark.parametrize("kind", KINDS)
def test_a_layer_from_prompts_to_tokens(dev, kind):
    B, prompts, steps = 5, (37, 1, 90, 16, 150), 3
    layer = Layer(kind, dev, 11, B, 200)
    t, r = layer.t, layer.r
    lens = np.array(prompts, np.int32)
    offsets = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    T = int(offsets[-1])
    x, h = bf16(ref.bf16_bits(r.standard_normal((T, D))), dev), bf16(ref.bf16_bits(2 * r.standard_normal((T, D))), dev)
    before = h.clone()
    got = layer.step(x, h, t(offsets), t(lens), total=int(lens.sum()))
    layer.check(got, x, before, h, offsets, lens)
    # the prompts' cache rows read back are the rows appended
    back = layer.M.mla_cache_read(t(offsets), layer.pool, layer.t_table, t(lens), kv_lora_rank=L, qk_rope=R, page_size=PS,
                                  total_rows=T, debug=True)
    req = np.repeat(np.arange(B), prompts)
    pos = np.arange(T) - offsets[req]
    row = layer.table[req, pos // PS].astype(np.int64) * PS + pos % PS
    assert np.array_equal(bits(back), bits(layer.pool).reshape(-1, L + R)[row])

    # one token a request, captured once; its inputs are filled in between replays
    one = np.arange(B + 1, dtype=np.int32)
    x1, h1 = torch.zeros(B, D, dtype=torch.bfloat16, device=dev), torch.zeros(B, D, dtype=torch.bfloat16, device=dev)
    t_one, t_lens = t(one), t(lens)
    layer.step_weight = t(layer.weight).expand(B, HI).contiguous()
    graph, seen = None, []
    for s in range(steps):
        lens = lens + 1
        xb, hb = ref.bf16_bits(r.standard_normal((B, D))), ref.bf16_bits(2 * r.standard_normal((B, D)))
        x1.copy_(bf16(xb, dev))
        h1.copy_(bf16(hb, dev))
        t_lens.copy_(t(lens))
        if s == 0:      # first eagerly, then the same step captured (the rows are written again, alike)
            eager = layer.step(x1, h1, t_one, t_lens)
            torch.cuda.synchronize()
            eager = {k: v.clone() for k, v in eager.items()}
            h1.copy_(bf16(hb, dev))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = layer.step(x1, h1, t_one, t_lens)
        graph.replay()
        torch.cuda.synchronize()
        layer.check(got, x1, bf16(hb, dev), h1, one, lens)
        if s == 0:
            assert all(np.array_equal(raw(got[k]), raw(eager[k])) for k in eager)
        seen.append(bits(got["y"]))
    assert not np.array_equal(seen[0], seen[1])
