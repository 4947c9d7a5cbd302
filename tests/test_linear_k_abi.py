"""CPU: mla_linear_fp8 and mla_linear_int8 take k up to 2^17, past which an fp32 sum's rounding would show in bf16."""
import pytest

from test_code_ops_abi import FAKE, TOO_SMALL, UNSUPPORTED, lib  # noqa: F401


@pytest.mark.parametrize("name", ["mla_linear_fp8", "mla_linear_int8"])
def test_longest_k(lib, name):  # noqa: F811
    def call(k, n=64, wsp_bytes=256):
        return getattr(lib, name)(2, n, k, FAKE, FAKE, FAKE, FAKE, FAKE, n, 0, FAKE, wsp_bytes, None)
    assert call((1 << 17) + 16) == UNSUPPORTED and call(1 << 20) == UNSUPPORTED
    # what is taken gets as far as the next check
    assert call(1 << 17, wsp_bytes=0) == TOO_SMALL and call(1 << 17, n=1 << 24, wsp_bytes=0) == TOO_SMALL
