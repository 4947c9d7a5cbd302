"""GPU: mla_rmsnorm_quant under any epsilon that it accepts, down to the smallest fp32 number, bit for bit.

A row of zeros has epsilon alone under its root, so a small one leaves fp32's range there (1 / epsilon
passes 2^128); the row is zeros all the same, its scale 1.  Rows of values are the others' check."""
import numpy as np
import pytest

import code_ref as cr
import latent_ref as ref
from test_rmsnorm_quant_gpu import FORMATS, check, dev  # noqa: F401

pytestmark = pytest.mark.gpu
EPSILONS = (1e-45, 1e-41, 1e-39, 2.9e-39, 2.0 ** -127, 2.0 ** -126, 1e-36, 2.0 ** -101, 2.0 ** -100, 1e-25, 2.0 ** -60, 1.0,
            2.0 ** 60, 1e30, 3e38)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D", [(9, 72), (9, 1304), (9, 8200), (1100, 1032)])   # a warp, a block, more a thread, warps
def test_rows_of_zeros_and_others(dev, fmt, T, D):  # noqa: F811
    r = np.random.default_rng(4)
    v = r.standard_normal((T, D))
    v[0], v[1], v[4] = 0.0, -0.0, 2.0 ** -133
    v[3] *= 2.0 ** -100
    v[5] = np.where(np.arange(D) % 9, 0.0, 1.0)
    v[T - 1] = 0.0
    x, g = ref.bf16_bits(v), ref.bf16_bits(r.standard_normal(D))
    for eps in EPSILONS:
        check(dev, FORMATS[fmt], x, None, g, eps=float(np.float32(eps)))
    h, y = cr.rmsnorm(x, None, g, float(np.float32(1e-45)))
    assert not (y[0] & 0x7FFF).any()
