"""The package on a torch that has only its public interface."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in dir(torch._C):
    if name.startswith("_cuda_"):
        delattr(torch._C, name)
import sliding_window_sparse_b200 as swa
import sliding_window_sparse_b200.seq_parallel
assert swa._raw_stream is swa._stream
assert swa._current_device is torch.cuda.current_device
"""


def test_import_without_private_cuda_calls():
    """A torch built without CUDA has no torch._C._cuda_*: the package and its CPU parts load."""
    res = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
