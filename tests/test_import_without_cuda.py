"""The package imports, and its C interface loads, where torch was built without CUDA.  CPU only."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# the names that a torch without CUDA lacks, taken away before the package is imported
CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import w8a8_dynamic_quant_gb300 as W
assert W._capi.lib().w8a8_version() >= 100
assert W.fp8_matmul_workspace_bytes(4, 256, 256) > 0
try:
    W.w8a8_fp8_quant(torch.zeros(2, 128, dtype=torch.bfloat16))
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise SystemExit("a tensor on the CPU was taken")
"""


def test_import_without_cuda():
    from w8a8_dynamic_quant_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
