"""Plain 64-bit numpy forms of the latent-cache operators, for their tests: the cache formats'
rows, and attention over a paged cache.  Nothing here uses the package."""
import math

import numpy as np

BF16, E4M3, E2M1 = 0, 1, 2
E2M1_GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3_grid():
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * np.exp2(e - 7.0))


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_bits(x):
    """float64 -> bf16 bits, one rounding (nearest, ties to even), by exact scaling."""
    x = np.asarray(x, np.float64)
    out = np.zeros(x.shape, np.uint16)
    fin = np.isfinite(x)
    a = np.where(fin, np.abs(x), 0.0)
    e = np.maximum(np.frexp(a)[1] - 1, -126)
    n = np.rint(np.ldexp(a, 7 - e)).astype(np.int64)          # 2^7 .. 2^8, or less below 2^-126
    mag = np.where(n >= 256, ((e + 1 + 127) << 7), np.where(n >= 128, ((e + 127) << 7) + (n - 128), n))
    mag = np.minimum(mag, 0x7F80)
    out[...] = mag
    out[np.isinf(x)] = 0x7F80
    out[np.isnan(x)] = 0x7FC0
    return out | (np.signbit(x) & ~np.isnan(x)).astype(np.uint16) << 15


def nearest_code(a, grid):
    """Index of the nearest value of an ascending grid, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(grid, a), 0, len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (hi % 2 == 0))
    return np.where(up | (a >= grid[hi]), hi, lo)


def least_exponent(amax, limit, low, high):
    """The least e in [low, high] with amax <= limit * 2^e; 0 for amax = 0."""
    out = np.zeros(amax.shape, np.int64)
    for i, v in np.ndenumerate(amax):
        if v == 0 or not np.isfinite(v):
            continue
        e = math.frexp(v)[1] - 12
        while v > math.ldexp(limit, e):
            e += 1
        out[i] = min(max(e, low), high)
    return out


def encode(y_bits, rope_bits, fmt):
    """Rows of bf16 bits [n, L], [n, R] -> (row bytes [n, bytes], row scales f32 or None)."""
    n, L = y_bits.shape
    y, rope = bf16_values(y_bits), np.ascontiguousarray(rope_bits).view(np.uint8)
    if fmt == BF16:
        return np.concatenate([np.ascontiguousarray(y_bits).view(np.uint8), rope], 1), None
    sign = np.signbit(y)
    if fmt == E4M3:
        bad = ~np.isfinite(y).all(1)
        e = least_exponent(np.abs(y).max(1), 448.0, -126, 127)
        e[bad] = 0
        with np.errstate(invalid="ignore"):
            code = nearest_code(np.ldexp(np.abs(y), -e[:, None]), e4m3_grid()).astype(np.uint8) | sign.astype(np.uint8) << 7
        code[bad] = 0x7F
        return np.concatenate([code, rope], 1), np.ldexp(1.0, e).astype(np.float32)
    g = y.reshape(n, L // 32, 32)
    bad = ~np.isfinite(g).all(2)
    e = least_exponent(np.abs(g).max(2), 7.0, -127, 127)
    e[bad] = 0
    with np.errstate(invalid="ignore"):
        code = nearest_code(np.ldexp(np.abs(g), -e[..., None]), E2M1_GRID).astype(np.uint8)
    code |= np.signbit(g).astype(np.uint8) << 3
    code[bad] = 0
    code = code.reshape(n, L)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    pad = np.zeros((n, -(L // 2 + L // 32) % 16), np.uint8)
    return np.concatenate([code[:, 0::2] | code[:, 1::2] << 4, scale, pad, rope], 1), None


def decode(rows, scales, fmt, L, R):
    """Row bytes (and row scales) -> the float64 values [n, L + R] that they stand for."""
    rope = bf16_values(np.ascontiguousarray(rows[:, -2 * R:]).view(np.uint16))
    if fmt == BF16:
        return np.concatenate([bf16_values(np.ascontiguousarray(rows[:, :2 * L]).view(np.uint16)), rope], 1)
    if fmt == E4M3:
        table = np.concatenate([e4m3_grid(), [np.nan]])
        c = table[rows[:, :L] & 127] * np.where(rows[:, :L] >> 7, -1.0, 1.0) * scales.astype(np.float64)[:, None]
    else:
        b = rows[:, :L // 2]
        code = np.stack([b & 15, b >> 4], -1).reshape(len(b), L)
        s = rows[:, L // 2:L // 2 + L // 32].astype(np.float64)
        s = np.where(s == 255, np.nan, np.exp2(s - 127))
        c = E2M1_GRID[code & 7] * np.where(code >> 3, -1.0, 1.0) * np.repeat(s, 32, 1)
    return np.concatenate([c, rope], 1)


def append(new, gamma, freqs, pos, eps, L, R, q=None, N=0):
    """bf16 bits of new rows [n, L + R] -> (latent bits, rope bits, turned q bits or None).
    Mean square and root in extended precision, each result rounded once."""
    x = bf16_values(new)
    c = x[:, :L].astype(np.longdouble)
    with np.errstate(all="ignore"):
        ms = (c * c).sum(1, keepdims=True) / L + np.longdouble(eps)
        y = c / np.sqrt(ms) * bf16_values(gamma).astype(np.longdouble)
        y = y.astype(np.float64)
    f = bf16_values(freqs)[pos]

    def turn(v, f):
        out = np.empty_like(v)
        with np.errstate(all="ignore"):
            out[..., 0::2] = v[..., 0::2] * f[..., 0::2] - v[..., 1::2] * f[..., 1::2]
            out[..., 1::2] = v[..., 0::2] * f[..., 1::2] + v[..., 1::2] * f[..., 0::2]
        return bf16_bits(out)

    q2 = None
    if q is not None:
        q2 = q.copy()
        q2[..., N:] = turn(bf16_values(q[..., N:]), f[:, None])
    return bf16_bits(y), turn(x[:, L:], f), q2


def visible(mask, window, length, pos):
    """Keys [lo, hi) of the query at `pos` in a request of `length` cached tokens."""
    if mask == 0:
        return 0, length
    hi = max(0, min(pos + 1, length))
    return (max(0, pos + 1 - window) if mask == 2 else 0), hi


def attention(q, w_uk, w_uv, rows, lens, offsets, scale, mask, window):
    """Latent attention in 64 bits, keys and values expanded.  q [T, H, N+R], w_uk [H, L, N],
    w_uv [H, V, L] values; rows[b] the values [len, L + R] of request b's cache.  A query
    that sees no key gets 0 and -inf; tokens behind the last request are left NaN."""
    T, H, _ = q.shape
    L, N = w_uk.shape[1:]
    out = np.full((T, H, w_uv.shape[1]), np.nan)
    lse = np.full((T, H), np.nan)
    for b, length in enumerate(lens):
        k = np.einsum("kl,hln->hkn", rows[b][:, :L], w_uk)
        v = np.einsum("kl,hvl->hkv", rows[b][:, :L], w_uv)
        n = int(offsets[b + 1]) - int(offsets[b])
        for i in range(n):
            t = int(offsets[b]) + i
            lo, hi = visible(mask, window, length, length - n + i)
            if hi <= lo:
                out[t], lse[t] = 0, -np.inf
                continue
            s = scale * ((k[:, lo:hi] @ q[t, :, :N, None])[..., 0] + q[t, :, N:] @ rows[b][lo:hi, L:].T)
            with np.errstate(invalid="ignore"):
                p = np.exp(s - s.max(1, keepdims=True))
                lse[t] = s.max(1) + np.log(p.sum(1))
                out[t] = ((p / p.sum(1, keepdims=True))[:, None] @ v[:, lo:hi])[:, 0]
    return out, lse
