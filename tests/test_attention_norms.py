"""The bound on rows' norms lets rounding pass and nothing else: checked on the oracle, without a GPU."""
import numpy as np
import pytest

from attention_check import U
from attention_norms import bound, rows_off
from oracle import attention_oracle as A

# (query tokens, keys, heads, key heads, head size, factor on q, scale): the shapes of the GPU tests, small to long
CASES = [(1, 2000, 8, 2, 128, 10.0, None), (70, 2000, 8, 2, 128, 10.0, 0.11), (40, 5000, 8, 1, 128, 1.0, None),
         (129, 1300, 3, 1, 64, 1.0, None), (4, 777, 4, 1, 128, 1.0, None)]
FORMATS = [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int8", "f16"), ("int4", "bf16"), ("int4", "f16")]


def rounded(x, dtype):
    """To nearest in bf16 or fp16 (normal range)."""
    if dtype == "f16":
        return x.astype(np.float16).astype(np.float64)
    b = x.astype(np.float32).view(np.uint32)
    b = (b + np.uint32(0x7FFF) + ((b >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)
    return b.view(np.float32).astype(np.float64)


def case(c, dtype, fmt, seed=1):
    lq, lk, h, kv, d, sharp, scale = c
    g = np.random.default_rng(seed)
    q = rounded(g.standard_normal((lq, h, d)) * sharp, dtype)
    k, v = (rounded(g.standard_normal((lk, kv, d)), dtype) for _ in range(2))
    if fmt in A.TOP:
        k, v = (A.read_back(*A.quantise(x.astype(np.float32), fmt)) for x in (k, v))
    return q, k, v, scale


def as_the_kernels_round(q, k, v, scale, dtype, fmt):
    """Attention with the roundings that the bound allows for, each to nearest."""
    d = q.shape[-1]
    scale = d**-0.5 if scale is None else scale
    quant = fmt in A.TOP
    if quant:
        hm = A.hadamard(d)
        q, k, v = (rounded(x, "f16") for x in (q @ hm * (8.0 / d), k @ hm / 8.0, v @ hm / 8.0))
    lq, h, _ = q.shape
    kv = k.shape[1]
    ok = A.seen(lq, k.shape[0], 0)
    out = np.zeros((lq, h, d))
    for i in range(h):
        s = np.where(ok, scale * (q[:, i] @ k[:, i * kv // h].T), -np.inf)
        w = np.exp(s - s.max(-1, keepdims=True))
        out[:, i] = rounded(w, "f16" if quant else dtype) @ v[:, i * kv // h] / w.sum(-1, keepdims=True)
    if quant:
        out = out @ hm * (8.0 / d)
    return rounded(out, dtype)


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("c", CASES)
def test_rounding_passes_and_lost_keys_do_not(c, fmt, dtype):
    q, k, v, scale = case(c, dtype, fmt)
    want, tol = bound(q, k, v, 0, scale, dtype, fmt)
    off = rows_off(as_the_kernels_round(q, k, v, scale, dtype, fmt), want, tol)
    assert off.max() <= 1.0
    assert (rows_off(np.zeros_like(want), want, tol) > 5.0).all()
    # the second half of the values lost; a tile of 64 values of the last 128 keys lost; two tiles' values swapped
    n = k.shape[0]
    half, tile, swap = v.copy(), v.copy(), v.copy()
    half[n // 2:] = 0.0
    tile[n - 128:n - 64] = 0.0
    swap[n - 128:n - 64], swap[n - 64:] = v[n - 64:], v[n - 128:n - 64]
    for lost in (half, tile, swap):
        bad = A.attention(q, k, lost, 0, scale)[0]
        off = rows_off(bad, want, tol)
        if c[5] == 1.0:  # of weights that are spread, most rows show it
            assert (off[-1] > 1.0).all() and np.mean(off > 1.0) > 0.5
        elif lost is half or c[0] > 16:  # a few sharp rows may have no weight in one tile
            assert off.max() > 1.0
    # one of two parts of the keys taken for the whole
    first = rows_off(A.attention(q, k[n // 2:], v[n // 2:], 0, scale)[0], want, tol)
    assert (first[-1] > 1.0).all() if c[5] == 1.0 else first.max() > 1.0  # a sharp row may lie wholly in one part


def test_units_are_half_an_ulp():
    x = np.linspace(1.0, 2.0, 4097)
    for dtype in ("bf16", "f16"):
        assert np.abs(rounded(x, dtype) - x).max() <= U[dtype]
