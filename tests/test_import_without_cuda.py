"""The package imports, and its host-side functions run, on a torch that was built without CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# a torch without CUDA has none of these
CODE = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream", "_cuda_getCurrentStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import mxfp8_activation_quant_gb300 as m
assert m.interleave_gate_up(torch.zeros(2, 3, 4), torch.ones(2, 3, 4)).shape == (12, 4)
assert m.moe_workspace_bytes(4, 2, 8, 512, 256) > 0 and m.sf_bytes(0, 4, 64) == 8
"""


def test_import_without_cuda():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
