"""Plain 64-bit numpy forms of the operators over 8-bit codes, for their tests.  Nothing here uses
the package."""
import numpy as np

import latent_ref as ref

NONE, E4M3, INT8 = 0, 1, 2
E4M3_VALUES = np.concatenate([ref.e4m3_grid(), [np.nan], -ref.e4m3_grid(), [np.nan]])


def nearest_e4m3(v):
    """float64 values within [-448, 448] -> e4m3 codes, nearest, ties to even."""
    return ref.nearest_code(np.abs(v), ref.e4m3_grid()).astype(np.uint8) | np.signbit(v).astype(np.uint8) << 7


def encode(y_bits, fmt):
    """Rows of bf16 bits [n, D] -> (codes uint8 [n, D], scales f32 [n]); a row with a NaN or an
    infinity gets NaN codes (e4m3) or zero codes and a NaN scale (int8)."""
    y = ref.bf16_values(y_bits)
    bad = ~np.isfinite(y).all(1)
    y = np.where(bad[:, None], 0.0, y)
    amax = np.abs(y).max(1)
    if fmt == E4M3:
        e = ref.least_exponent(amax, 448.0, -126, 127)
        codes = nearest_e4m3(np.ldexp(y, -e[:, None]))
        codes[bad] = 0x7F
        return codes, np.ldexp(1.0, e).astype(np.float32)
    scale = np.where(amax > 0, np.maximum(amax.astype(np.float32) * (np.float32(1) / np.float32(127)), np.float32(2.0 ** -126)),
                     np.float32(1)).astype(np.float32)
    codes = np.rint(y / scale[:, None].astype(np.float64)).astype(np.int8).view(np.uint8)
    scale[bad] = np.nan
    return codes, scale


def rmsnorm(x, residual, gamma, eps):
    """bf16 bits -> (bits of h, bits of y); the root in extended precision, each result rounded once."""
    h = x
    with np.errstate(all="ignore"):
        if residual is not None:
            h = ref.bf16_bits(ref.bf16_values(x) + ref.bf16_values(residual))
        if gamma is None:
            return h, h
        c = ref.bf16_values(h).astype(np.longdouble)
        ms = (c * c).sum(1, keepdims=True) / c.shape[1] + np.longdouble(eps)
        return h, ref.bf16_bits((c / np.sqrt(ms) * ref.bf16_values(gamma).astype(np.longdouble)).astype(np.float64))


def layer_norm(x, gamma, beta, eps):
    c = ref.bf16_values(x).astype(np.longdouble)
    with np.errstate(all="ignore"):
        d = c - c.mean(1, keepdims=True)
        y = d / np.sqrt((d * d).mean(1, keepdims=True) + np.longdouble(eps))
        y = y * ref.bf16_values(gamma).astype(np.longdouble) + ref.bf16_values(beta).astype(np.longdouble)
    return ref.bf16_bits(y.astype(np.float64))


def turn(x, f):
    """Pairs of the last axis of bf16 bits x turned by the (cos, sin) bits of f, rounded once."""
    x, f = ref.bf16_values(x), ref.bf16_values(f)
    out = np.empty(np.broadcast_shapes(x.shape, f.shape))
    with np.errstate(all="ignore"):
        out[..., 0::2] = x[..., 0::2] * f[..., 0::2] - x[..., 1::2] * f[..., 1::2]
        out[..., 1::2] = x[..., 0::2] * f[..., 1::2] + x[..., 1::2] * f[..., 0::2]
    return ref.bf16_bits(out)


class Pages:
    """Seeded requests over pages in random order: their tables and where each token's row is (-1: nowhere)."""

    def __init__(self, seed, ps, qlens, past, spare=2):
        r = self.rng = np.random.default_rng(seed)
        B, self.ps, self.T = len(qlens), ps, int(sum(qlens))
        self.lens = np.array([a + b for a, b in zip(qlens, past)], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        pages = -(-self.lens // ps)
        order = r.permutation(int(pages.sum()) + spare).astype(np.int32)
        self.table = np.full((B, max(1, int(pages.max()))), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        self.num_pages, self.rows = len(order), len(order) * ps
        self.req = np.repeat(np.arange(B), qlens)
        self.pos = np.concatenate([np.arange(n - k, n) for k, n in zip(qlens, self.lens)]).astype(np.int64)
        self.place()

    def place(self):
        """Anew after a change of the table, the lengths or pos."""
        inside = (self.pos >= 0) & (self.pos < self.table.shape[1] * self.ps)
        p = np.where(inside, self.pos, 0)
        page = self.table[self.req, p // self.ps].astype(np.int64)
        good = inside & (page >= 0) & (page < self.num_pages)
        self.row = np.where(good, page * self.ps + p % self.ps, -1)
