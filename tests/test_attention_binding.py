"""The binding of the rotary, cache and attention calls, as far as it goes without a GPU."""
import os
import subprocess
import sys

import pytest

from exl3_trellis_quantized_gb300 import binding as B

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


@pytest.fixture
def on_cpu(monkeypatch):
    """Checks of arguments without the demand for a GPU (no call of the library is reached)."""
    monkeypatch.setattr(B, "_need", lambda t, dtype, name: None)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_cache_addresses_stay_those_of_its_tensors(on_cpu, fmt):
    cache = B.KVCache.empty(3, 16, 2, 64, fmt, device="cpu")
    other = B.KVCache.empty(3, 16, 2, 64, fmt, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale", "fmt", "head_dim", "args"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(other, name))
    for name in ("k", "v", "k_scale", "v_scale"):
        t = getattr(cache, name)
        assert getattr(cache.args, name) == (None if t is None else t.data_ptr())
    assert (cache.num_pages, cache.kv_heads, cache.page_size, cache.head_dim, cache.fmt) == (3, 2, 16, 64, fmt)
