"""The package is imported, and refuses host tensors, on a torch without CUDA bindings."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_cuda_bindings_of_torch():
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import moe_decode_ffn_gb300 as m
for f in (lambda: m.si_quantize_mxfp4(torch.zeros(4, 64)), lambda: m.si_moe_sort(torch.zeros(2, 2, dtype=torch.int32), 4)):
    try:
        f()
    except ValueError as e:
        assert "CUDA" in str(e), e
    else:
        raise AssertionError("taken")
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
