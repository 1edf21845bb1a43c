"""The package imports with a PyTorch that was built without CUDA, whose C module
lacks the CUDA functions: its host-only parts are of use there."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda")]:
    delattr(torch._C, name)
import w4a8_quantized_linear_gb300 as cider
from w4a8_quantized_linear_gb300 import inputs, column_parallel
assert callable(cider._raw_stream)
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda device: Stream if device == 3 else None
assert cider._raw_stream(3) == 77
"""


def test_import():
    done = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
