"""The binding of the rotary, cache and attention calls, as far as it goes without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

from exl3_trellis_quantized_gb300 import binding as B

FAKE = 1 << 20  # an aligned address that is never followed
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


def touched(t):
    """Addresses of a view's elements."""
    at = torch.zeros((), dtype=torch.int64)
    for n, st in zip(t.shape, t.stride()):
        at = at.unsqueeze(-1) + torch.arange(n) * st
    return set((t.data_ptr() + t.element_size() * at.flatten()).tolist())


def test_overlap_of_views():
    """No overlap is missed, and views side by side in a fused projection's rows are not taken for one."""
    x = torch.zeros(10, 6, 8, dtype=torch.bfloat16)
    h = torch.zeros(6, 10, 8, dtype=torch.bfloat16).transpose(0, 1)  # heads outermost
    flat = x.view(-1)
    views = [x[:, :2], x[:, 2:4], x[:, 4:], x[:, 1:3], x[3:, :2], x[:3, 2:], x[9:, :], x[:1, 5:], x[2:2], x, flat[:96], flat[96:112],
             flat[24:48], flat[8:40].view(2, 2, 8), x[::2, :3], x[1::2, 3:], h, h[:, :3], h[:, 3:], h[:4, 2:], h[4:, 2:], h[:4]]
    for a in views:
        for b in views:
            assert B._overlap(a, b) == B._overlap(b, a)
            if touched(a) & touched(b):
                assert B._overlap(a, b)
    for a, b in ((0, 1), (0, 2), (1, 2), (4, 1), (6, 4 - 4), (16, 0), (17, 18), (12, 7)):
        if not touched(views[a]) & touched(views[b]):
            assert not B._overlap(views[a], views[b]), (a, b)


def test_unknown_layout_is_a_value_error(on_cpu):
    positions, phases = torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int64)
    with pytest.raises(ValueError):
        B._rope_args(positions, phases, "neox", 1.0, 2)
    assert B._rope_args(positions, phases, "half", 1.0, 2).rot_dim == 16


def test_tensors_of_one_call_lie_on_one_device(monkeypatch):
    """Told apart before any address reaches a kernel (the meta device stands in for a second GPU)."""
    reached = []
    monkeypatch.setattr(B, "_need", lambda t, dtype, name: None)
    monkeypatch.setattr(B, "_heads", lambda t, dtype, name: B._Heads(FAKE, 128, 64))
    monkeypatch.setattr(B, "_out_like", lambda x, out, name: (x, B._Heads(FAKE, 128, 64)))
    monkeypatch.setattr(B, "_raw_stream", lambda index: None)
    monkeypatch.setattr(B, "_workspace_bytes", lambda *sizes: 16)

    class Library:
        def __getattr__(self, name):
            return lambda *args: reached.append(name) or 0

    monkeypatch.setattr(B, "lib", lambda: Library())

    def ints(*shape, dtype=torch.int32, device="cpu"):
        return torch.zeros(shape, dtype=dtype, device=device)

    def rows(device="cpu"):
        return torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=device)

    cache = B.KVCache.empty(3, 16, 2, 64, "int8", device="cpu")
    far = B.KVCache.empty(3, 16, 2, 64, "int8", device="meta")
    calls = {
        "rope": (lambda x, p, f: B.rope(x, p, f), [rows(), ints(2), ints(32, dtype=torch.int64)]),
        "kv_write": (lambda c, k, v, s, q, p, f: B.kv_write(c, k, v, s, q=q, positions=p, phases=f),
                     [cache, rows(), rows(), ints(2, dtype=torch.int64), rows(), ints(2), ints(32, dtype=torch.int64)]),
        "kv_read": (lambda c, s, k, v: B.kv_read(c, s, k=k, v=v), [cache, ints(2, dtype=torch.int64), rows(), rows()]),
        "attention_prompt": (lambda q, k, v, cu: B.attention_prompt(q, k, v, cu), [rows(), rows(), rows(), ints(2)]),
        "attention_paged": (lambda q, c, t, cu, n, w: B.attention_paged(q, c, t, cu, n, 1, 1, workspace=w),
                            [rows(), cache, ints(1, 3), ints(2), ints(1), ints(64, dtype=torch.uint8)]),
    }
    for name, (call, args) in calls.items():
        reached.clear()
        call(*args)
        assert reached == ["exl3_" + name]
        for i, t in enumerate(args):
            other = list(args)
            other[i] = far if t is cache else t.to("meta")
            reached.clear()
            with pytest.raises(ValueError, match="device"):
                call(*other)
            assert not reached
    with pytest.raises(ValueError, match="device"):
        B.KVCache(cache.k, far.v, cache.k_scale, cache.v_scale, "int8")
