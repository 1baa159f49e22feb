"""The package imports, and its calls find their stream, on a torch without the private accessors that the binding
prefers.  CPU only; in a process of its own, since the names are taken away before the import."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import mamba_selective_scan_03_amd as jscan
from mamba_selective_scan_03_amd import _binding as b

torch.cuda.current_stream = lambda i: type("S", (), {"cuda_stream": 1000 + i})
assert b._raw_stream(3) == 1003 and b._current_device is torch.cuda.current_device
assert callable(jscan.prefill) and callable(jscan.gated_scan)
print("imported")
"""


def test_import_without_private_accessors():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "imported", r.stderr
