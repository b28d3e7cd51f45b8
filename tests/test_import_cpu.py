"""The package imports where torch lacks its private names for the current
stream and device (a build without GPU support): argument checks and size
queries need no GPU."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import w8a8_int8_quantized_amd as w8
assert w8.moe_workspace_bytes(4, 2, 256, 256) > 0
try:
    w8.norm_residual_quant(torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(128, dtype=torch.bfloat16))
except w8.W8Error:
    print("refused")
"""


def test_import_without_torch_private_names():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "refused" in r.stdout
