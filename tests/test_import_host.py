"""The package imports, and its host functions work, on a torch build without CUDA."""
import subprocess
import sys

from conftest import ROOT

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import mla_decode_attention_06_gb300 as M
assert M.mla_cache_row_bytes(M.MLA_CACHE_E2M1, 512, 64) == 400
try:
    M.mla_rmsnorm_quant(torch.zeros(2, 64, dtype=torch.bfloat16))
except ValueError:
    print("refused")
"""


def test_import_without_cuda():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
