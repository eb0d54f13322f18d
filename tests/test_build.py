"""The build script by itself."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_TORCH = r"""
import importlib.util, os, sys
sys.modules["torch"] = None              # importing it raises ImportError
spec = importlib.util.spec_from_file_location("build", os.path.join("long_context_paged_gb300", "build.py"))
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
path = b.build()
assert os.path.exists(path) and path == b.LIB
"""


def test_the_library_builds_without_pytorch():
    """The C library needs nvcc alone; only the binding's fast path needs PyTorch's headers, and is left
    out, with a word about it."""
    from long_context_paged_gb300 import build as b
    b.build()
    before = os.path.getmtime(b.FAST)
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "fast path was not built" in r.stderr
    assert os.path.getmtime(b.FAST) == before
