"""GPU: int8 codes that mla_rmsnorm_quant wrote into byte buffers go into mla_linear_int8 as they are, as e4m3
codes go into mla_linear_fp8."""
import pytest
import torch

from test_linear_gpu import codes, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 20, 64, 300])
def test_codes_as_bytes(dev, T):  # noqa: F811
    import mla_decode_attention_06_gb300 as M
    g = torch.Generator(device=dev).manual_seed(T)
    x = torch.randn(T, 512, generator=g, device=dev).to(torch.bfloat16)
    w, ws = codes("int8", 3, 264, 512, dev)
    raw = torch.empty(T, 512, dtype=torch.uint8, device=dev)
    got, s, _ = M.mla_rmsnorm_quant(x, code_format=M.MLA_CODES_INT8, codes_out=raw)
    assert got is raw
    want = M.mla_linear_int8(raw.view(torch.int8), s, w, ws)
    assert torch.equal(M.mla_linear_int8(raw, s, w, ws), want)
    assert torch.equal(M.mla_linear_int8(raw, s, w.view(torch.uint8), ws, debug=True), want)
