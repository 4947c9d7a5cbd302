"""Cases that measure the 8-bit operators around the attention: normalisation with codes out, the
projections over codes, the indexer's cache write, and the latent cache read back.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits, in 64
where a rounding border decides a stored code) or, with ``own``, through the package's public entry
points.  ``exact`` evaluates the definitions in 64 bits.

  norm    h = bf16(x + residual); y = bf16(h / sqrt(mean(h^2) + eps) * gamma); codes of y with one
          scale a token: int8, scale amax / 127; e4m3, the least 2^e with amax <= 448 * 2^e
  linear  out[t, n] = bf16(x_scale[t] * w_scale[n] * sum_k x[t, k] * w[n, k]), codes int8 or e4m3
  index   the indexer's keys: LayerNorm, rotation of the last R values, e4m3 codes with one power of
          two a row, written into the paged cache; its queries: rotation, codes, scale * weight
  read    rows of the paged latent cache (bf16, e4m3, e2m1) as bf16 values, request after request

A token i of a request with q tokens sits at position len - q + i of its cache.
"""
import math
import random

import torch

own = False

EPS = 1e-6
FORMATS = ("bf16", "e4m3", "e2m1")
DEV = "cuda"


# ------------------------------------------------------------------------------- cases

def _norm(name, codes, T, D, pad=0, residual=True, gamma=True):
    return dict(name=name, op="norm", codes=codes, T=T, D=D, pad=pad, residual=residual, gamma=gamma)


def _linear(name, codes, T, N, K):
    return dict(name=name, op="linear", codes=codes, T=T, N=N, K=K)


def _index(name, B, q_lo, q_hi, past, H, D, R, ps, ln=True):
    return dict(name=name, op="index", B=B, q_lo=q_lo, q_hi=q_hi, past=past, H=H, D=D, R=R, ps=ps, ln=ln, draw=1)


def _read(name, fmt, B, q_lo, q_hi, past, ps, narrow=False):
    return dict(name=name, op="read", fmt=fmt, B=B, q_lo=q_lo, q_hi=q_hi, past=past, ps=ps, narrow=narrow, draw=1)


def listed():
    return [
        # one conversation's next token enters a layer: latency alone
        _norm("norm e4m3 one token", "e4m3", 1, 8192),
        # a decode batch's query latents, a slice of the fused down projection [1536 + 576]
        _norm("norm int8 query latents of 64", "int8", 64, 1536, pad=576, residual=False),
        # a prefill step's residual stream before a projection
        _norm("norm e4m3 prompts", "e4m3", 8192, 8192),
        # the fused down projection of one token: latency, and few rows of weights a multiprocessor
        _linear("linear int8 one token", "int8", 1, 2112, 8192),
        # a decode batch's queries out of their latents, 128 heads of 192
        _linear("linear e4m3 batch of 64", "e4m3", 64, 24576, 1536),
        # a ragged batch through the output projection of 128 heads of 128
        _linear("linear int8 ragged batch", "int8", 333, 8192, 16384),
        # prompts: queries out of their latents
        _linear("linear int8 prompts", "int8", 4096, 24576, 1536),
        # prompts: the output projection
        _linear("linear e4m3 prompts", "e4m3", 8192, 8192, 16384),
        # a decode step of a full batch: one key a request, 64 index heads
        _index("index batch of 64", 64, 1, 1, 4000, 64, 128, 64, 64),
        # prompts of a prefill step
        _index("index prompts", 5, 300, 3100, 0, 64, 128, 64, 64),
        # a cached prefix of one conversation handed on
        _read("read e2m1 one prefix", "e2m1", 1, 4000, 4000, 0, 64),
        # a batch's e4m3 cache read back, 16-row pages
        _read("read e4m3 batch", "e4m3", 48, 1000, 8000, 0, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "index", "read"))
    ps = rng.choice((8, 16, 32, 64, 128))
    if op == "norm":
        D = 8 * _log(rng, 8, 2048)
        T = _log(rng, 1, max(1, min(16384, 8192 * 8192 // D)))
        c = _norm("", rng.choice(("e4m3", "int8", "bf16")), T, D, rng.choice((0, 0, 8, 64, 576)), rng.random() < 0.6,
                  rng.random() < 0.8)
    elif op == "linear":
        N, K = 8 * _log(rng, 8, 3000), 16 * _log(rng, 4, 1024)
        T = _log(rng, 1, max(1, min(8192, 8192 * 8192 * 16384 // (N * K))))
        c = _linear("", rng.choice(("int8", "e4m3")), T, N, K)
    elif op == "index":
        B = _log(rng, 1, 128)
        q_hi = _log(rng, 1, max(1, 8000 // B))
        D = rng.choice((64, 128, 128, 96))
        c = _index("", B, rng.randint(1, q_hi), q_hi, rng.randint(0, 9000), rng.choice((1, 4, 17, 32, 64)), D,
                   rng.choice((0, 32, 64)), ps, rng.random() < 0.7)
    else:
        B = _log(rng, 1, 128)
        q_hi = _log(rng, 1, max(1, 250000 // B))
        c = _read("", rng.choice(FORMATS), B, rng.randint(1, q_hi), q_hi, rng.choice((0, 0, rng.randint(1, 5000))), ps,
                  rng.random() < 0.2)
    if op in ("index", "read"):
        c["draw"] = rng.randint(2, 1 << 20)
    del c["name"]
    return c


def _widths(case):   # latent and rope width
    return (64, 16) if case["narrow"] else (512, 64)


def _lengths(case):
    """(new or read tokens, cached tokens) of every request: the case alone decides them."""
    r = random.Random(case["draw"] * 1000003 + case["B"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    return q, [n + (r.randint(case["past"] // 2, case["past"]) if case["past"] else 0) for n in q]


def _row_bytes(fmt, L, R):
    if fmt == "bf16":
        return 2 * (L + R)
    if fmt == "e4m3":
        return L + 2 * R
    return -(-(L // 2 + L // 32) // 16) * 16 + 2 * R


def work(case):
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        out = 2 * D if case["codes"] == "bf16" else D + 4
        n = T * (2 * D + out + (4 * D if case["residual"] else 0)) + (2 * D if case["gamma"] else 0)
        return {"bytes": n, "flops": T * D * 6}
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * K + N * K + 4 * (T + N) + 2 * T * N, "flops": 2 * T * N * K}
    q, lens = _lengths(case)
    T = sum(q)
    tables = 4 * sum((n - 1) // case["ps"] - (n - k) // case["ps"] + 1 for k, n in zip(q, lens))
    if case["op"] == "index":
        D, H, R = case["D"], case["H"], case["R"]
        return {"bytes": T * (3 * D + 4 + H * (3 * D + 8) + 2 * R) + tables, "flops": T * (H + 1) * (4 * D + 3 * R)}
    L, R = _widths(case)
    row = _row_bytes(case["fmt"], L, R) + (4 if case["fmt"] == "e4m3" else 0)
    return {"bytes": T * (row + 2 * (L + R)) + tables, "flops": T * L}


# ------------------------------------------------------------------------------- formats

def _to_bf16(x):
    """float64 -> bf16, rounded once (nearest even): through float32 rounded to odd."""
    f = x.float()
    f = torch.where(f.double().abs() > x.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    odd = (f.double() != x) & torch.isfinite(f)
    return (f.view(torch.int32) | odd.int()).view(torch.float32).to(torch.bfloat16)


def _quant_e4m3(y):
    """Rows of bf16 values -> (codes, the least power of two a row with amax <= 448 scale)."""
    v = y.float()
    f, x = torch.frexp(v.abs().amax(-1))
    e = torch.where(f > 0, (x - 9 + (f > 0.875).int()).clamp(-126, 127), 0)
    scale = torch.exp2(e.double()).float()
    return (v.double() / scale.double()[..., None]).float().to(torch.float8_e4m3fn), scale


def _quant_int8(y):
    """Rows of bf16 values -> (codes, amax / 127 rounded to 32 bits)."""
    v = y.float()
    amax = v.abs().amax(-1)
    scale = torch.where(amax > 0, (amax / 127).clamp_min(2.0 ** -126), 1.0)
    return torch.round(v.double() / scale.double()[..., None]).to(torch.int8), scale


def _values(rows, scales, fmt, L, R, dtype):
    """Cache rows [n, bytes] (and row scales [n]) -> the values [n, L + R] they stand for."""
    if fmt == "bf16":
        return rows.view(torch.bfloat16).to(dtype)
    rope = rows[..., -2 * R:].contiguous().view(torch.bfloat16).to(dtype)
    if fmt == "e4m3":
        c = rows[..., :L].contiguous().view(torch.float8_e4m3fn).to(dtype) * scales[..., None].to(dtype)
    else:
        b = rows[..., :L // 2].int()
        code = torch.stack((b & 15, b >> 4), -1).flatten(-2)
        m, x = code & 1, (code >> 1) & 3
        mag = torch.where(x == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(x.to(dtype) - 1)).to(dtype)
        s = torch.exp2(rows[..., L // 2:L // 2 + L // 32].to(dtype) - 127)
        c = torch.where(code > 7, -mag, mag) * s.repeat_interleave(32, -1)
    return torch.cat((c, rope), -1)


# ------------------------------------------------------------------------------- inputs

def _paged(case, s, g):
    """Pages of all requests in random order, three more than they fill, and where tokens go."""
    q, lens = _lengths(case)
    B, ps = case["B"], case["ps"]
    counts = [-(-n // ps) for n in lens]
    order = torch.randperm(sum(counts) + 3, generator=g, device=DEV).int()
    table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    s.update(T=sum(q), q_lens=q, lens=lens, table=table, rows=(at + 3) * ps,
             offsets=torch.tensor([0] + q, device=DEV).cumsum(0).int(),
             cache_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    bf = torch.bfloat16
    s = dict(case=case)
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        # a few channels carry values far above the others'
        s["x"] = (normal(T, D + case["pad"]) * torch.exp(0.5 * normal(D + case["pad"]))).to(bf)[:, :D]
        s["residual"] = (4 * normal(T, D)).to(bf) if case["residual"] else None
        s["gamma"] = (1 + 0.1 * normal(D)).to(bf) if case["gamma"] else None
        s["h"] = torch.empty(T, D, dtype=bf, device=DEV) if case["residual"] else None
        return s
    if case["op"] == "linear":
        for k, rows, size in (("x", case["T"], 1.0), ("w", case["N"], case["K"] ** -0.5)):
            v = (normal(rows, case["K"]) * size).to(bf)
            if case["codes"] == "int8":
                s[k], s[k + "_scale"] = _quant_int8(v)
            else:   # weights come with a scale of their own making, not a power of two
                s[k], sc = _quant_e4m3(v)
                s[k + "_scale"] = sc if k == "x" else sc * (1 + 0.5 * torch.rand(rows, generator=g, device=DEV))
        return s
    _paged(case, s, g)
    T = s["T"]
    if case["op"] == "index":
        H, D, R = case["H"], case["D"], case["R"]
        s["k_new"] = (1.5 * normal(T, D) + 0.3).to(bf)
        s["q"] = normal(T, H, D).to(bf)
        s["weight"] = normal(T, H) / math.sqrt(H * D)
        s["gamma"], s["beta"] = ((1 + 0.1 * normal(D)).to(bf), (0.1 * normal(D)).to(bf)) if case["ln"] else (None, None)
        s["freqs"] = None
        if R:
            ang = torch.arange(max(s["lens"]), device=DEV, dtype=torch.float64)[:, None] * \
                10000.0 ** (-2.0 * torch.arange(R // 2, device=DEV, dtype=torch.float64) / R)
            s["freqs"] = torch.stack((ang.cos(), ang.sin()), -1).flatten(-2).to(bf)
        pool = torch.randint(0, 127, (s["rows"], D), generator=g, device=DEV, dtype=torch.uint8)
        s["pool"] = pool.view(torch.float8_e4m3fn)
        s["scales"] = torch.rand(s["rows"], generator=g, device=DEV)
        s["q_codes"] = torch.empty(T, H, D, dtype=torch.float8_e4m3fn, device=DEV)
        s["q_scales"] = torch.empty(T, H, device=DEV)
        return s
    L, R = _widths(case)
    n, fmt = s["rows"], case["fmt"]
    rope = normal(n, R).to(bf).view(torch.uint8)
    s["scales"] = None
    if fmt == "bf16":
        s["pool"] = torch.cat((normal(n, L).to(bf).view(torch.uint8), rope), -1)
    elif fmt == "e4m3":
        codes, _ = _quant_e4m3(normal(n, L).to(bf))
        s["scales"] = 0.01 * torch.exp(normal(n))
        s["pool"] = torch.cat((codes.view(torch.uint8), rope), -1)
    else:
        codes = torch.randint(0, 256, (n, L // 2), generator=g, device=DEV, dtype=torch.uint8)
        sc = torch.randint(123, 129, (n, L // 32), generator=g, device=DEV, dtype=torch.uint8)
        pad = torch.zeros(n, -(L // 2 + L // 32) % 16, dtype=torch.uint8, device=DEV)
        s["pool"] = torch.cat((codes, sc, pad, rope), -1)
    s["out"] = torch.empty(T, L + R, dtype=bf, device=DEV)
    return s


# ------------------------------------------------------------------------------- plain forms

def _places(s):
    """Position and physical row of every token of the call."""
    T = torch.arange(s["T"], device=DEV)
    req = torch.searchsorted(s["offsets"][1:].long(), T, right=True)
    pos = s["cache_lens"].long()[req] - s["offsets"].long()[req + 1] + T
    ps = s["case"]["ps"]
    return pos, s["table"].long()[req, pos // ps] * ps + pos % ps


def _turn(x, f):
    """Pairs of x turned by the (cos, sin) pairs of f, in 64 bits."""
    x, f = x.double().unflatten(-1, (-1, 2)), f.double().unflatten(-1, (-1, 2))
    return torch.stack((x[..., 0] * f[..., 0] - x[..., 1] * f[..., 1],
                        x[..., 0] * f[..., 1] + x[..., 1] * f[..., 0]), -1).flatten(-2)


def _plain_norm(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    y = h
    if s["gamma"] is not None:   # 64 bits: the last bit of a bf16 value can decide a stored code
        d = h.double()
        y = _to_bf16(d / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS) * s["gamma"].double())
    got = {} if s["residual"] is None else {"h": h}
    if s["case"]["codes"] == "bf16":
        return {**got, "y": y.clone()}
    codes, scales = (_quant_int8 if s["case"]["codes"] == "int8" else _quant_e4m3)(y)
    return {**got, "codes": codes, "scales": scales}


def _plain_linear(s):
    out = torch.matmul(s["x"].float(), s["w"].float().T)
    return {"out": (out * s["x_scale"][:, None] * s["w_scale"]).to(torch.bfloat16)}


def _plain_index(s):
    D, R = s["case"]["D"], s["case"]["R"]
    pos, row = _places(s)
    k, q = s["k_new"], s["q"]
    if s["gamma"] is not None:
        d = k.double()
        d = d - d.mean(-1, keepdim=True)
        k = _to_bf16(d / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS) * s["gamma"].double() + s["beta"].double())
    if R:
        f = s["freqs"][pos]
        k = torch.cat((k[:, :D - R], _to_bf16(_turn(k[:, D - R:], f))), -1)
        q = torch.cat((q[..., :D - R], _to_bf16(_turn(q[..., D - R:], f[:, None]))), -1)
    codes, scale = _quant_e4m3(k)
    s["pool"].view(torch.uint8)[row] = codes.view(torch.uint8)
    s["scales"][row] = scale
    q_codes, scale = _quant_e4m3(q)
    return {"k": s["pool"], "k_scales": s["scales"], "q": q_codes, "q_scales": scale * s["weight"]}


def _plain_read(s):
    L, R = _widths(s["case"])
    _, row = _places(s)
    sc = None if s["scales"] is None else s["scales"][row]
    # 64 bits: a code times a scale has more bits than 32-bit arithmetic keeps
    return {"rows": _to_bf16(_values(s["pool"][row], sc, s["case"]["fmt"], L, R, torch.float64))}


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "linear": _plain_linear, "index": _plain_index, "read": _plain_read}[case["op"]](s)
    import mla_decode_attention_06_gb300 as M
    if case["op"] == "norm":
        fmt = {"bf16": M.MLA_CODES_BF16, "e4m3": M.MLA_CODES_E4M3, "int8": M.MLA_CODES_INT8}[case["codes"]]
        out, scales, h = M.mla_rmsnorm_quant(s["x"], s["gamma"], epsilon=EPS, code_format=fmt, residual=s["residual"],
                                             residual_out=s["h"])
        got = {} if h is None else {"h": h}
        return {**got, "y": out} if case["codes"] == "bf16" else {**got, "codes": out, "scales": scales}
    if case["op"] == "linear":
        fn = M.mla_linear_int8 if case["codes"] == "int8" else M.mla_linear_fp8
        return {"out": fn(s["x"], s["x_scale"], s["w"], s["w_scale"])}
    if case["op"] == "index":
        M.mla_indexer_append(s["k_new"], s["offsets"], s["pool"], s["scales"], s["table"], s["cache_lens"],
                             page_size=case["ps"], freqs_cis=s["freqs"], k_norm_gamma=s["gamma"], k_norm_beta=s["beta"],
                             epsilon=EPS, q=s["q"], q_weight=s["weight"], q_codes=s["q_codes"], q_scales=s["q_scales"])
        return {"k": s["pool"], "k_scales": s["scales"], "q": s["q_codes"], "q_scales": s["q_scales"]}
    L, R = _widths(case)
    fmt = (M.MLA_CACHE_BF16, M.MLA_CACHE_E4M3, M.MLA_CACHE_E2M1)[FORMATS.index(case["fmt"])]
    return {"rows": M.mla_cache_read(s["offsets"], s["pool"], s["table"], s["cache_lens"], kv_lora_rank=L, qk_rope=R,
                                     page_size=case["ps"], cache_format=fmt, kv_scales=s["scales"], out=s["out"])}


# ------------------------------------------------------------------------------- 64 bits

def _exact_e4m3(y):
    """The e4m3 values nearest y / unit and the unit, a row's least power of two that holds it."""
    amax = y.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax / 448)      # by exponents: a logarithm can miss a power of two by a bit
    unit = torch.where(amax > 0, torch.exp2((e - (m == 0.5).int()).clamp(-126, 127).double()), 1.0)
    a = y / unit
    step = torch.exp2((torch.frexp(a)[1].clamp_min(-5) - 4).double())
    return torch.round(a / step) * step, unit[..., 0]


def _exact_norm(s):
    h = s["x"].double()
    got = {}
    if s["residual"] is not None:
        h = h + s["residual"].double()
        got["h"] = h
        h = _to_bf16(h).double()     # what follows sees the bf16 row
    y = h
    if s["gamma"] is not None:
        y = s["gamma"].double() * h * (h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS).pow(-0.5)
    if s["case"]["codes"] == "bf16":
        return {**got, "y": y}
    y = _to_bf16(y).double()         # the codes are those of the bf16 row
    if s["case"]["codes"] == "e4m3":
        codes, scales = _exact_e4m3(y)
        return {**got, "codes": codes, "scales": scales}
    scales = y.abs().amax(-1) / 127
    return {**got, "codes": torch.round(y / scales.float().double()[:, None]), "scales": scales}


def _exact_index(s):
    case = s["case"]
    D, R = case["D"], case["R"]
    pos = torch.cat([torch.arange(n - k, n, device=DEV) for k, n in zip(s["q_lens"], s["lens"])])
    req = torch.repeat_interleave(torch.arange(case["B"], device=DEV), torch.tensor(s["q_lens"], device=DEV))
    row = s["table"][req, pos // case["ps"]].long() * case["ps"] + pos % case["ps"]
    k, q = s["k_new"].double(), s["q"].double()
    if s["gamma"] is not None:
        mean = k.sum(-1, keepdim=True) / D
        k = (k - mean) * s["gamma"].double() / ((k - mean).pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() + s["beta"].double()
        k = _to_bf16(k).double()     # the normalised row is a bf16 row
    if R:
        cs = s["freqs"][pos].double()
        turn = torch.complex(cs[:, 0::2].contiguous(), cs[:, 1::2].contiguous())

        def rotated(x, z):
            pairs = torch.view_as_complex(x[..., D - R:].reshape(*x.shape[:-1], R // 2, 2).contiguous())
            return torch.cat((x[..., :D - R], _to_bf16(torch.view_as_real(pairs * z).flatten(-2)).double()), -1)

        k, q = rotated(k, turn), rotated(q, turn[:, None])
    pool, scales = s["pool"].double(), s["scales"].double()
    pool[row], scales[row] = _exact_e4m3(k)
    codes, unit = _exact_e4m3(q)
    return {"k": pool, "k_scales": scales, "q": codes, "q_scales": unit * s["weight"].double()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "linear":
        x = s["x"].double() * s["x_scale"].double()[:, None]
        return {"out": x @ (s["w"].double() * s["w_scale"].double()[:, None]).T}
    if case["op"] == "index":
        return _exact_index(s)
    L, R = _widths(case)
    rows = []
    for b, (n, length) in enumerate(zip(s["q_lens"], s["lens"])):
        j = torch.arange(length - n, length, device=DEV)
        rows.append(s["table"][b].long()[j // case["ps"]] * case["ps"] + j % case["ps"])
    row = torch.cat(rows)
    raw = s["pool"][row]
    if case["fmt"] != "e2m1":
        return {"rows": _values(raw, None if s["scales"] is None else s["scales"][row], case["fmt"], L, R, torch.float64)}
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV, dtype=torch.float64)
    nibbles = torch.stack((raw[:, :L // 2] % 16, raw[:, :L // 2] // 16), -1).long()
    unit = torch.pow(2.0, raw[:, L // 2:L // 2 + L // 32].double() - 127)
    c = (grid[nibbles].reshape(len(row), L // 32, 32) * unit[..., None]).reshape(len(row), L)
    return {"rows": torch.cat((c, raw[:, -2 * R:].contiguous().view(torch.bfloat16).double()), -1)}
