"""GPU: mla_rmsnorm_quant at the lower end of bf16's range, bit for bit: results next to half its least number,
of values and gammas whose product fp32 does not hold, beside ordinary values of the same row."""
import numpy as np
import pytest

import code_ref as cr
import latent_ref as ref
from test_rmsnorm_quant_gpu import FORMATS, check, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D", [(4000, 8), (1200, 512), (40, 1304), (20, 8200)])
def test_results_about_the_least_number(dev, fmt, T, D):  # noqa: F811
    """Every eighth value 2^-k, so 1 / sqrt is some 2^(k + 1.5); the others' products with gamma some 2^-134 less that."""
    r = np.random.default_rng(D)
    eps = float(np.float32(1e-30))
    k = r.integers(0, 18, (T, 1))
    e = r.integers(-55, -30, (1, D))
    g = r.uniform(1, 2, (1, D)) * np.exp2(e)
    g[:, ::8] = 1.0
    v = r.choice([-1, 1], (T, D)) * r.uniform(1, 2, (T, D)) * np.exp2(-136.0 - k - e + r.integers(-2, 4, (T, D)))
    v[:, ::8] = np.exp2(-k)
    v[r.random((T, D)) < 0.1] = 0.0
    g[:, 5] = 0.0
    x, g = ref.bf16_bits(v), ref.bf16_bits(g[0])
    check(dev, FORMATS[fmt], x, None, g, eps=eps)
    y = cr.rmsnorm(x, None, g, eps)[1] & 0x7FFF
    assert ((y > 0) & (y < 4)).sum() > T * D // 8          # they are where the test wants them


@pytest.mark.parametrize("fmt", FORMATS)
def test_zeros_among_values(dev, fmt):  # noqa: F811
    """Rows of nothing but zeros, of mostly zeros, and zeros of gamma, both signs: zeros with the product's sign."""
    r = np.random.default_rng(2)
    v = np.where(r.random((1300, 264)) < r.random((1300, 1)), 0.0, r.standard_normal((1300, 264)))
    v *= r.choice([-1, 1], v.shape)
    g = np.where(r.random(264) < 0.3, 0.0, r.standard_normal(264)) * r.choice([-1, 1], 264)
    check(dev, FORMATS[fmt], ref.bf16_bits(v), None, ref.bf16_bits(g))
    check(dev, FORMATS[fmt], ref.bf16_bits(v[:50]), ref.bf16_bits(-v[:50]), ref.bf16_bits(g))
