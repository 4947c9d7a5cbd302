"""GPU: the LayerNorm of mla_indexer_append where keys equal their row's mean, bit for bit.

Such a key's deviation is zero, so the result is beta: for a beta of zero a zero, and for a row of equal
keys a row of zeros under scale 1, for every head dimension (only some have a reciprocal that fp32 holds).
Keys next to the mean leave a deviation of the row's last bits."""
import numpy as np
import pytest

import code_ref as cr
import latent_ref as ref
from test_indexer_append_gpu import EPS, Case, check, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def case(D, rows, beta):
    c = Case(D=D, H=0, R=0, ps=16, qlens=(len(rows),))
    c.k = ref.bf16_bits(rows)
    if not beta:
        c.beta = np.zeros_like(c.beta)
    return c


@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("D", [8, 24, 40, 64, 72, 88, 96, 104, 120, 128, 136, 152, 168, 184, 200, 232, 248, 256])
def test_equal_keys(dev, D, beta):  # noqa: F811
    top = (1 + np.arange(128) / 128)[:, None] * np.exp2(np.arange(128) % 20 - 10)[:, None]
    c = case(D, np.concatenate([top, -top]).repeat(D, 1), beta)
    check(c, dev)
    if not beta:
        y = cr.layer_norm(c.k, c.gamma, c.beta, EPS)
        assert not (y & 0x7FFF).any()


@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("D", [40, 72, 96, 104, 136, 184, 248, 256])
def test_keys_at_and_next_to_the_mean(dev, D, beta):  # noqa: F811
    r = np.random.default_rng(D)
    n = 60
    base = ref.bf16_values(ref.bf16_bits(r.uniform(1.1, 1.9, (n, 1)) * np.exp2(r.integers(-6, 7, (n, 1)))))
    step = np.exp2(np.floor(np.log2(base)) - 7)
    off = r.integers(-1, 2, (n, D // 2)) * step
    at = np.stack([base + off, base - off], -1).reshape(n, D)          # the mean is base, as many keys are
    near = np.ones((20, D))
    near[:, -2] = 2.0
    near[:, -1] = np.exp2(-np.arange(20.0))                              # ones next to a mean of 1 + 2^-i / D
    check(case(D, np.concatenate([at, near]), beta), dev)
