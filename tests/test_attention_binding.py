"""The binding of the rotary, cache and attention calls, as far as it goes without a GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_without_torchs_private_stream_call():
    """A torch that lacks the call (one built without CUDA, or a later one) still imports the package."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "import exl3_trellis_quantized_gb300 as E\n"
            "assert callable(E.rope)\n")
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
