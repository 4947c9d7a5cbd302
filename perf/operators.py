"""Cases that measure the latent-cache operators: append, 4-bit decode, expanded prefill.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits, in
64 where a rounding border decides a stored code) or, with ``own``, through the package's
public entry points.  ``exact`` evaluates the definitions in 64 bits.

Shapes: H heads, N no-rope and R rope columns of a query, latent width L, value width V, page
size ps.  The widths are the package's own: (N, R, L, V) = (128, 64, 512, 128), and the narrow
(32, 16, 64, 32).  A query token i of a request with q tokens sits at position len - q + i.
"""
import math
import random

import torch

own = False

WIDE = dict(N=128, R=64, L=512, V=128)
NARROW = dict(N=32, R=16, L=64, V=32)
EPS = 1e-6
MASKS = {"null": 0, "causal": 1, "window": 2}
FORMATS = ("bf16", "e4m3", "e2m1")
DEV = "cuda"


# ------------------------------------------------------------------------------- cases

def _append(name, fmt, B, q_lo, q_hi, past, H, ps, narrow=False):
    return dict(name=name, op="append", fmt=fmt, B=B, q_lo=q_lo, q_hi=q_hi, past=past, H=H, ps=ps,
                mask="causal", window=0, narrow=narrow, draw=1)


def _decode(name, B, q, lo, hi, H, ps, mask="causal", window=0, narrow=False):
    return dict(name=name, op="decode", fmt="e2m1", B=B, q_lo=q, q_hi=q, lo=lo, hi=hi, H=H, ps=ps,
                mask=mask, window=window, narrow=narrow, draw=1)


def _prefill(name, fmt, B, q_lo, q_hi, past, H, ps, mask="causal", window=0, narrow=False):
    return dict(name=name, op="prefill", fmt=fmt, B=B, q_lo=q_lo, q_hi=q_hi, past=past, H=H, ps=ps,
                mask=mask, window=window, narrow=narrow, draw=1)


def listed():
    return [
        # one conversation's next token enters a 4-bit cache: latency alone
        _append("append e2m1 one token", "e2m1", 1, 1, 1, 1000, 128, 64),
        # a decode step of a full batch, one token a request
        _append("append bf16 batch of 64", "bf16", 64, 1, 1, 4000, 128, 64),
        # speculative decoding: one to three tokens a request, 16-row pages
        _append("append e4m3 few tokens each", "e4m3", 33, 1, 3, 700, 16, 16),
        # prompts of a prefill step written in one call, queries of all heads turned
        _append("append e2m1 prompts", "e2m1", 5, 300, 3100, 0, 128, 64),
        # the narrow widths, two requests: the smallest decode
        _decode("decode e2m1 narrow", 2, 1, 37, 70, 4, 16, narrow=True),
        # a serving step: 64 requests of 1k to 8k tokens
        _decode("decode e2m1 batch of 64", 64, 1, 1024, 8192, 128, 64),
        # long contexts, few requests: the keys have to be split over the device
        _decode("decode e2m1 long", 8, 1, 32768, 131072, 128, 64),
        # two speculative tokens, a sliding window, a tensor-parallel share of the heads
        _decode("decode e2m1 window", 19, 2, 3000, 20000, 16, 32, mask="window", window=4096),
        # ragged short prompts, all heads
        _prefill("prefill bf16 short prompts", "bf16", 7, 1, 500, 0, 128, 64),
        # one long prompt on a tensor-parallel share of the heads
        _prefill("prefill bf16 long prompt", "bf16", 1, 16384, 16384, 0, 16, 64),
        # a chunk of two requests behind a cached 4-bit context
        _prefill("prefill e2m1 chunk", "e2m1", 2, 500, 520, 7600, 128, 64),
        # prompts over an e4m3 cache with e4m3 weights
        _prefill("prefill e4m3 prompts", "e4m3", 3, 1500, 2300, 0, 128, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill"))
    narrow = rng.random() < 0.15
    H = rng.choice((1, 4, 16, 24, 64, 127, 128))
    ps = rng.choice((8, 16, 32, 64, 128))
    mask = rng.choice(("causal", "causal", "null", "window"))
    window = _log(rng, 1, 5000) if mask == "window" else 0
    if op == "append":
        B = _log(rng, 1, 128)
        q_hi = _log(rng, 1, max(1, 8000 // B))
        c = _append("", rng.choice(FORMATS), B, rng.randint(1, q_hi), q_hi, rng.randint(0, 9000), H, ps, narrow)
    elif op == "decode":
        B = _log(rng, 1, 64)
        hi = _log(rng, 3, min(131072, 500000 // B))
        q = rng.choice((1, 1, 1, 2, 3))
        c = _decode("", B, q, rng.randint(q, max(q, hi)), max(q, hi), H, ps, mask, window, narrow)
    else:
        B = _log(rng, 1, 9)
        q_hi = _log(rng, 1, 6000)
        past = rng.choice((0, 0, _log(rng, 1, 9000)))
        while B * H * q_hi * (q_hi + past) > 3e9 or B * (q_hi + past) > 20000:
            q_hi, past = max(1, q_hi * 2 // 3), past * 2 // 3
        c = _prefill("", rng.choice(FORMATS), B, rng.randint(1, q_hi), q_hi, past, H, ps, mask, window, narrow)
    c["draw"] = rng.randint(2, 1 << 20)
    del c["name"]
    return c


def _widths(case):
    return NARROW if case["narrow"] else WIDE


def _lengths(case):
    """(query tokens, cached tokens) of every request: the case alone decides them."""
    r = random.Random(case["draw"] * 1000003 + case["B"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    if case["op"] == "decode":
        return q, [max(n, r.randint(case["lo"], case["hi"])) for n in q]
    return q, [n + (r.randint(case["past"] // 2, case["past"]) if case["past"] else 0) for n in q]


def _row_bytes(fmt, L, R):
    if fmt == "bf16":
        return 2 * (L + R)
    if fmt == "e4m3":
        return L + 2 * R
    return -(-(L // 2 + L // 32) // 16) * 16 + 2 * R


def _pairs(case):
    """(query, key) pairs that the mask leaves, and the keys that some query attends."""
    pairs = keys = 0
    W = case["window"]
    for n, length in zip(*_lengths(case)):
        p0 = length - n
        if case["mask"] == "null":
            pairs, keys = pairs + n * length, keys + length
        elif case["mask"] == "causal":
            pairs, keys = pairs + n * p0 + n * (n + 1) // 2, keys + length
        else:
            pairs += sum(min(p0 + i + 1, W) for i in range(n))
            keys += length - max(0, p0 + 1 - W)
    return pairs, keys


def work(case):
    w, H, fmt = _widths(case), case["H"], case["fmt"]
    N, R, L, V = w["N"], w["R"], w["L"], w["V"]
    q, lens = _lengths(case)
    T = sum(q)
    row = _row_bytes(fmt, L, R) + (4 if fmt == "e4m3" else 0)
    if case["op"] == "append":
        # new rows in, cache rows and their values out, queries in and out, the rotations
        n = T * (2 * (L + R) + row + 2 * (L + R) + 4 * H * (N + R) + 2 * R)
        return {"bytes": n, "flops": T * (6 * L + 6 * R * (H + 1) // 2)}
    pairs, keys = _pairs(case)
    tables = sum(-(-n // case["ps"]) * 4 for n in lens)
    wb = H * L * (N + V) * (1 if case["op"] == "prefill" and fmt == "e4m3" else 2)
    n = keys * row + tables + wb + 2 * T * H * (N + R + V)
    if case["op"] == "decode":   # absorbed: the query and the output pass through the latent space
        flops = 2 * T * H * L * (N + V) + 2 * pairs * H * (2 * L + R)
    else:                        # expanded: every cached row becomes H keys and values
        flops = 2 * keys * H * L * (N + V) + 2 * pairs * H * (N + R + V)
    return {"bytes": n, "flops": flops}


# ------------------------------------------------------------------------------- formats

def _to_bf16(x):
    """float64 -> bf16, rounded once (nearest even): through float32 rounded to odd."""
    f = x.float()
    f = torch.where(f.double().abs() > x.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    odd = (f.double() != x) & torch.isfinite(f)
    return (f.view(torch.int32) | odd.int()).view(torch.float32).to(torch.bfloat16)


def _exponent(amax, over, low, high):
    """The smallest e with amax <= 0.875 * 2^(e + over), within [low, high]; 0 where amax is 0."""
    f, x = torch.frexp(amax)
    e = (x - over + (f > 0.875).int()).clamp(low, high)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _quant_e4m3(y):
    """Rows of bf16 values -> (codes, power-of-two row scale with amax <= 448 scale)."""
    v = y.float()
    e = _exponent(v.abs().amax(-1), 9, -126, 127)
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return (v.double() / scale.double()[..., None]).float().to(torch.float8_e4m3fn), scale


def _quant_e2m1(y):
    """Rows of bf16 values -> (packed codes, low nibble first; e8m0 scale bytes of 32 values)."""
    v = y.double().unflatten(-1, (-1, 32))
    e = _exponent(v.abs().amax(-1).float(), 3, -127, 127)
    a = v.abs() * torch.ldexp(torch.ones_like(e, dtype=torch.float64), -e)[..., None]
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    code = (code + 8 * torch.signbit(v).int()).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), (e + 127).to(torch.uint8)


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

def prepare(case, seed):
    w, H, B, ps, fmt = _widths(case), case["H"], case["B"], case["ps"], case["fmt"]
    N, R, L, V = w["N"], w["R"], w["L"], w["V"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    bf = torch.bfloat16
    q, lens = _lengths(case)
    T = sum(q)
    stride = -(-max(lens) // ps)
    pages = sum(-(-n // ps) for n in lens)
    order = torch.randperm(pages + 3, generator=g, device=DEV).int()
    table = torch.full((B, stride), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        n = -(-lens[b] // ps)
        table[b, :n] = order[at:at + n]
        at += n
    offsets = torch.tensor([0] + q, device=DEV).cumsum(0).int()
    rows = (pages + 3) * ps
    s = dict(case=case, T=T, q_lens=q, lens=lens, table=table, offsets=offsets, total=sum(lens),
             cache_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), scales=None,
             q=normal(T, H, N + R).to(bf))
    if case["op"] == "append":
        # the new rows are a slice of the fused down projection's output
        s["new"] = (normal(T, 2 * L + L + R) * 1.7).to(bf)[:, 2 * L:]
        ang = torch.arange(max(lens), device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-2.0 * torch.arange(R // 2, device=DEV, dtype=torch.float64) / R)
        s["freqs"] = torch.stack((ang.cos(), ang.sin()), -1).flatten(-2).to(bf)
        s["gamma"] = (1 + 0.1 * normal(L)).to(bf)
        s["pool"] = torch.randint(0, 256, (rows, _row_bytes(fmt, L, R)), generator=g, device=DEV, dtype=torch.uint8)
        if fmt == "e4m3":
            s["scales"] = torch.rand(rows, generator=g, device=DEV)
        s["q_out"] = torch.empty_like(s["q"])
        s["rows_out"] = torch.empty(T, L + R, dtype=bf, device=DEV)
        return s
    c = normal(rows, L)
    c = (c * torch.rsqrt(c.square().mean(-1, keepdim=True))).to(bf)
    rope = normal(rows, R).to(bf).view(torch.uint8)
    if fmt == "bf16":
        s["pool"] = torch.cat((c.view(torch.uint8), rope), -1)
    elif fmt == "e4m3":
        codes, s["scales"] = _quant_e4m3(c)
        s["pool"] = torch.cat((codes.view(torch.uint8), rope), -1)
    else:
        codes, sc = _quant_e2m1(c)
        pad = torch.zeros(rows, -(L // 2 + L // 32) % 16, dtype=torch.uint8, device=DEV)
        s["pool"] = torch.cat((codes, sc, pad, rope), -1)
    s["w_uk"] = normal(H, L, N) / math.sqrt(N)
    s["w_uv"] = normal(H, V, L) / math.sqrt(L)
    for k in ("w_uk", "w_uv"):
        if case["op"] == "prefill" and fmt == "e4m3":
            x = s[k]
            na, nb = -(-x.shape[1] // 128), -(-x.shape[2] // 128)
            sc = x.abs().amax((1, 2), keepdim=True).expand(H, na, nb) / 448 * \
                (1 + 0.5 * torch.rand(H, na, nb, generator=g, device=DEV))
            s[k + "_scale"] = sc.contiguous()
            s[k] = (x / _blocks(sc, x)).to(torch.float8_e4m3fn)
        else:
            s[k] = s[k].to(bf)
    return s


def _blocks(scale, x):
    """128 x 128 block scales spread over the matrix that they scale."""
    return scale.repeat_interleave(128, 1)[:, :x.shape[1]].repeat_interleave(128, 2)[:, :, :x.shape[2]]


def _weights(s, dtype):
    return tuple(s[k].to(dtype) * _blocks(s[k + "_scale"], s[k]).to(dtype) if k + "_scale" in s else s[k].to(dtype)
                 for k in ("w_uk", "w_uv"))


# ------------------------------------------------------------------------------- plain forms

def _places(s):
    """Request, position and physical row of every query token."""
    T = torch.arange(s["T"], device=DEV)
    req = torch.searchsorted(s["offsets"][1:].long(), T, right=True)
    pos = s["cache_lens"].long()[req] - s["offsets"].long()[req + 1] + T
    ps = s["case"]["ps"]
    return req, pos, s["table"].long()[req, pos // ps] * ps + pos % ps


def _turn(x, f):
    """Pairs of x turned by the (cos, sin) pairs of f, in 64 bits."""
    x, f = x.double().unflatten(-1, (-1, 2)), f.double().unflatten(-1, (-1, 2))
    return torch.stack((x[..., 0] * f[..., 0] - x[..., 1] * f[..., 1],
                        x[..., 0] * f[..., 1] + x[..., 1] * f[..., 0]), -1).flatten(-2)


def _plain_append(s):
    case, w = s["case"], _widths(s["case"])
    N, R, L, fmt = w["N"], w["R"], w["L"], case["fmt"]
    _, pos, row = _places(s)
    f = s["freqs"][pos]
    c = s["new"][:, :L].double()
    # 64 bits: the last bit of a bf16 value can decide a stored code
    y = _to_bf16(c / torch.sqrt(c.square().mean(-1, keepdim=True) + EPS) * s["gamma"].double())
    rope = _to_bf16(_turn(s["new"][:, L:], f))
    s["q_out"][..., :N] = s["q"][..., :N]
    s["q_out"][..., N:] = _to_bf16(_turn(s["q"][..., N:], f[:, None]))
    rb = rope.view(torch.uint8)
    if fmt == "bf16":
        new = torch.cat((y.view(torch.uint8), rb), -1)
    elif fmt == "e4m3":
        codes, scale = _quant_e4m3(y)
        s["scales"][row] = scale
        new = torch.cat((codes.view(torch.uint8), rb), -1)
    else:
        codes, scale = _quant_e2m1(y)
        pad = torch.zeros(len(row), -(L // 2 + L // 32) % 16, dtype=torch.uint8, device=DEV)
        new = torch.cat((codes, scale, pad, rb), -1)
    s["pool"][row] = new
    s["rows_out"].copy_(_values(new, s["scales"][row] if fmt == "e4m3" else None, fmt, L, R, torch.float32))
    return _append_outputs(s)


def _append_outputs(s):
    got = {"pool": s["pool"], "q": s["q_out"], "rows": s["rows_out"]}
    if s["scales"] is not None:
        got["scales"] = s["scales"]
    return got


def _padded(s, dtype):
    """Keys [B, K, L + R], queries [B, Q, H, N + R], the mask [B, Q, K] and where each query sits."""
    case, w = s["case"], _widths(s["case"])
    ps, R, L = case["ps"], w["R"], w["L"]
    B, K, Q = case["B"], max(s["lens"]), max(s["q_lens"])
    j = torch.arange(K, device=DEV)
    live = j < s["cache_lens"][:, None]
    row = torch.where(live, s["table"].long()[:, j // ps] * ps + j % ps, 0)
    keys = _values(s["pool"][row], None if s["scales"] is None else s["scales"][row], case["fmt"], L, R, dtype)
    keys = torch.where(live[..., None], keys, 0)
    i = torch.arange(Q, device=DEV)
    n = s["offsets"].diff()[:, None]
    t = torch.where(i < n, s["offsets"][:-1, None] + i, 0).long()
    pos = (s["cache_lens"][:, None] - n + i)[..., None]
    see = live[:, None, :] & (i < n)[..., None]
    if case["mask"] != "null":
        see = see & (j <= pos)
    if case["mask"] == "window":
        see = see & (j > pos - case["window"])
    return keys, s["q"][t].to(dtype), see, (i < n), t


def _attend(score, see):
    """Softmax weights over the last axis where `see`; a row that sees nothing gets zeros."""
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1, total)


def _plain_attention(s):
    case, w = s["case"], _widths(s["case"])
    N, R, L = w["N"], w["R"], w["L"]
    scale = 1 / math.sqrt(N + R)
    uk, uv = _weights(s, torch.float32)
    keys, q, see, real, t = _padded(s, torch.float32)
    c, rope = keys[..., :L], keys[..., L:]
    if case["op"] == "decode":   # absorbed
        ql = torch.cat((torch.einsum("bqhn,hln->bqhl", q[..., :N], uk), q[..., N:]), -1)
        score = torch.matmul(ql.flatten(1, 2), keys.transpose(1, 2)).unflatten(1, (-1, case["H"])) * scale
        p = _attend(score, see[:, :, None])
        out = torch.einsum("bqhl,hvl->bqhv", torch.matmul(p.flatten(1, 2), c).view(*ql.shape[:3], L), uv)
    else:                        # expanded
        k = torch.einsum("bkl,hln->bhkn", c, uk)
        v = torch.einsum("bkl,hvl->bhkv", c, uv)
        qt = q.transpose(1, 2)
        score = torch.matmul(qt[..., :N], k.transpose(-1, -2))
        score += torch.matmul(qt[..., N:], rope[:, None].transpose(-1, -2))
        out = torch.matmul(_attend(score.mul_(scale), see[:, None]), v).transpose(1, 2)
    return {"out": out[real].to(torch.bfloat16)}


def run(state):
    s, case = state, state["case"]
    if not own:
        return _plain_append(s) if case["op"] == "append" else _plain_attention(s)
    import mla_decode_attention_06_gb300 as M
    ps = case["ps"]
    if case["op"] == "append":
        fmt = (M.MLA_CACHE_BF16, M.MLA_CACHE_E4M3, M.MLA_CACHE_E2M1)[FORMATS.index(case["fmt"])]
        M.mla_cache_append(s["new"], s["offsets"], s["pool"], s["table"], s["cache_lens"], s["freqs"], s["gamma"],
                           page_size=ps, epsilon=EPS, cache_format=fmt, kv_scales=s["scales"], q=s["q"],
                           q_out=s["q_out"], rows_out=s["rows_out"])
        return _append_outputs(s)
    kw = dict(page_size=ps, mask=MASKS[case["mask"]], window=case["window"])
    head = (s["q"], s["offsets"], s["pool"])
    tail = (s["table"], s["cache_lens"], s["w_uk"], s["w_uv"])
    if case["op"] == "decode":
        out, _ = M.mla_decode_paged_fp4(*head, *tail, **kw)
    elif case["fmt"] == "bf16":
        out, _ = M.mla_prefill_paged(*head, *tail, total_keys=s["total"], **kw)
    elif case["fmt"] == "e2m1":
        out, _ = M.mla_prefill_paged_fp4(*head, *tail, total_keys=s["total"], **kw)
    else:
        out, _ = M.mla_prefill_paged_fp8(*head, s["scales"], *tail[:3], s["w_uk_scale"], s["w_uv"],
                                         s["w_uv_scale"], total_keys=s["total"], **kw)
    return {"out": out}


# ------------------------------------------------------------------------------- 64 bits

def _exact_append(s):
    case, w = s["case"], _widths(s["case"])
    N, R, L, fmt = w["N"], w["R"], w["L"], case["fmt"]
    pos = torch.cat([torch.arange(n - k, n, device=DEV) for k, n in zip(s["q_lens"], s["lens"])])
    cs = s["freqs"][pos].double()
    turn = torch.complex(cs[:, 0::2].contiguous(), cs[:, 1::2].contiguous())

    def rotated(x):
        z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], R // 2, 2).contiguous())
        return torch.view_as_real(z * (turn if x.dim() == 2 else turn[:, None])).flatten(-2)

    x = s["new"].double()
    c = x[:, :L]
    y = c * s["gamma"].double() * (c.pow(2).sum(-1, keepdim=True) / L + EPS).pow(-0.5)
    got = {"pool": None, "q": torch.cat((s["q"][..., :N].double(), rotated(s["q"][..., N:])), -1)}
    scales = None
    if fmt != "bf16":
        y = _to_bf16(y).double()     # the stored codes are those of the bf16 row
        group = L if fmt == "e4m3" else 32
        z = y.reshape(-1, L // group, group)
        amax = z.abs().amax(-1, keepdim=True)
        # the smallest power of two that brings the largest magnitude to 448 (to 7)
        unit = torch.exp2(torch.ceil(torch.log2(amax / (448 if fmt == "e4m3" else 7))))
        bits, low = (3, -6) if fmt == "e4m3" else (1, 0)
        a = z / unit
        step = torch.exp2(torch.floor(torch.log2(a.abs().clamp_min(2.0 ** low))) - bits)
        v = torch.round(a / step) * step
        y = (v.clamp(-6, 6) if fmt == "e2m1" else v).mul(unit).reshape(-1, L)
        if fmt == "e4m3":
            scales = s["scales"].double()
            scales[_places(s)[2]] = unit.reshape(-1)
    got["rows"] = torch.cat((y, rotated(s["new"][:, L:]) if fmt == "bf16" else
                             _to_bf16(rotated(s["new"][:, L:])).double()), -1)
    if scales is not None:
        got["scales"] = scales
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    w = _widths(case)
    N, R, L, V = w["N"], w["R"], w["L"], w["V"]
    # few queries of a request: through the latent space, the same sums in another order
    latent = [n * (N + V) * 2 < length for n, length in zip(s["q_lens"], s["lens"])]
    if 2 * case["H"] * sum(n * m * (2 * L + R) if a else m * (n * (N + R + V) + L * (N + V))
                           for a, n, m in zip(latent, s["q_lens"], s["lens"])) > 8e12:
        return None
    uk, uv = _weights(s, torch.float64)
    out = torch.zeros(s["T"], case["H"], V, dtype=torch.float64, device=DEV)
    t = 0
    for b, (n, length) in enumerate(zip(s["q_lens"], s["lens"])):
        j = torch.arange(length, device=DEV)
        row = s["table"][b].long()[j // case["ps"]] * case["ps"] + j % case["ps"]
        x = _values(s["pool"][row], None if s["scales"] is None else s["scales"][row], case["fmt"], L, R,
                    torch.float64)
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        hide = torch.zeros(n, length, dtype=torch.bool, device=DEV)
        if case["mask"] != "null":
            hide |= j > pos
        if case["mask"] == "window":
            hide |= j <= pos - case["window"]
        q = s["q"][t:t + n].double()
        if latent[b]:
            ql = torch.einsum("qhn,hln->qhl", q[..., :N], uk)
            score = torch.einsum("qhl,kl->qhk", torch.cat((ql, q[..., N:]), -1), x)
            p = torch.softmax((score / math.sqrt(N + R)).masked_fill(hide[:, None], -math.inf), -1)
            out[t:t + n] = torch.einsum("qhl,hvl->qhv", torch.einsum("qhk,kl->qhl", p, x[:, :L]), uv)
        else:
            for h in range(case["H"]):
                score = q[:, h, :N] @ (x[:, :L] @ uk[h]).T + q[:, h, N:] @ x[:, L:].T
                p = torch.softmax((score / math.sqrt(N + R)).masked_fill(hide, -math.inf), -1)
                out[t:t + n, h] = p @ (x[:, :L] @ uv[h].T)
        t += n
    return {"out": out}
