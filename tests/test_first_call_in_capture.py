"""A program may capture its first call of the library: what the library sets up on first use (its scratch memory, its
kernels) can be set up inside a capture."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("first", ["fp4", "int8"])
def test_first_call_in_capture(first):
    r = subprocess.run([sys.executable, "-m", "tests.first_calls_captured", first], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
