"""CPU: the int8 scale of codes against its definition by division, for every bf16 value."""
import numpy as np

import code_ref as cr
import latent_ref as ref


def test_int8_scale_is_the_quotient_within_a_step():
    """max|y| * fl32(1 / 127) for max|y| / 127: the reciprocal and the product are each off by half a step at most,
    together by one of the quotient's, and the least scale is 2^-126."""
    mag = np.arange(1, 0x7F80, dtype=np.uint16)                     # all positive finite bf16 values
    rows = np.zeros((len(mag), 8), np.uint16)
    rows[:, 3] = mag
    rows[1::2, 3] |= 0x8000
    codes, scale = cr.encode(rows, cr.INT8)
    q = ref.bf16_values(mag).astype(np.float64) / 127
    want = q.astype(np.float32)
    normal = q >= 2.0 ** -126
    off = np.abs(scale.view(np.int32) - want.view(np.int32))
    assert (off[normal] <= 1).all() and off[normal].any()
    assert (scale[~normal] == np.float32(2.0 ** -126)).all()
    assert (np.abs(codes.view(np.int8)[normal, 3]) == 127).all()
    assert (cr.encode(np.zeros((1, 8), np.uint16), cr.INT8)[1] == 1).all()
