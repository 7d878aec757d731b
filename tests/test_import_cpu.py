"""The package imports, and its host-side calls work, on a torch without the private names that the operators'
bindings take for speed (in a process of its own: the names are gone before the package is imported)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
for name in {gone!r}:
    delattr(torch._C, name)
import sparse_moe_layer_gemm_amd as moe
assert moe.moe_mxfp4_scale_stride(160) == 8
seen = []
torch.cuda.current_device = lambda: 3
torch.cuda.current_stream = lambda device=None: seen.append(device) or type("S", (), dict(cuda_stream=77))()
assert moe._current_device() == 3 and moe._raw_stream(3) == 77 and seen == [3]
calls = []
moe._run("f", lambda *a: calls.append(a) or 0, 3, None, 5)
moe._run("f", lambda *a: calls.append(a) or 0, 3, 99, 6)
assert calls == [(5, 77), (6, 99)], calls
"""


@pytest.mark.parametrize("gone", [["_cuda_getCurrentRawStream", "_cuda_getDevice"]])
def test_import_without_private_torch_names(gone):
    r = subprocess.run([sys.executable, "-c", CODE.format(gone=gone)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
