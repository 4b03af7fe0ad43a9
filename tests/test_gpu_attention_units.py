"""Paged attention over quantised caches whose rows differ in size: the fp16 operands' units follow them.

Rows are held in norm (attention_norms): every entry of an operand within 2^-11 of itself, whatever the other rows are."""
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from attention_norms import assert_rows, bound
from oracle import attention_oracle as A
from test_gpu_attention import DEV, DT, cu, f64

pytestmark = pytest.mark.gpu


def run(q, k, v, fmt, page=32, window=0):
    """One sequence's last rows q over rows k, v (bf16) of a quantised cache, against the rows read back."""
    n, kv, dim = k.shape
    pages = (n + page - 1) // page
    cache = E.KVCache.empty(pages, page, kv, dim, fmt)
    E.kv_write(cache, k.to(DEV), v.to(DEV), torch.arange(n, device=DEV))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    got = E.attention_paged(q.to(DEV), cache, table, cu([q.shape[0]]), lens, q.shape[0], n, window=window)
    torch.cuda.synchronize()
    assert E.device_status() == 0
    kk, vv = (A.read_back(*A.quantise(t.float().numpy(), fmt)) for t in (k, v))
    dtype = "bf16" if q.dtype == torch.bfloat16 else "f16"
    want, tol = bound(q.double().numpy(), kk, vv, window, None, dtype, fmt)
    assert_rows(f64(got), want, tol, f"{q.shape[0]} queries over {n} keys")


def rows(n, kv, dim, sizes, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, kv, dim), generator=g)
    return (x * torch.as_tensor(sizes, dtype=torch.float32).view(-1, 1, 1)).to(torch.bfloat16)


def queries(n, heads, dim, dtype, by=1.0, seed=3):
    return (torch.randn((n, heads, dim), generator=torch.Generator().manual_seed(seed)) * by).to(DT[dtype])


# query tokens, keys, query heads, key heads: single tokens, a joint item, two halves, parts of the keys
SHAPES = [(1, 400, 8, 2), (40, 400, 8, 2), (150, 400, 8, 2), (24, 3000, 8, 1)]


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("int8", "f16"), ("int4", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("ratio", [1e4, 1e-4, 3e6, 1e-7])
def test_later_tiles_of_another_size(fmt, dtype, dim, shape, which, ratio):
    """The first 128 rows of one size, later ones larger or smaller."""
    q_len, n, heads, kv = shape
    sizes = torch.ones(n)
    sizes[128:] = ratio
    sizes = sizes / max(1.0, ratio) * (1.0 if which == "k" else 50.0)
    q = queries(q_len, heads, dim, dtype)
    k = rows(n, kv, dim, sizes if which == "k" else torch.ones(n), 1)
    v = rows(n, kv, dim, sizes if which == "v" else torch.ones(n), 2)
    run(q, k, v, fmt)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("q_len,heads", [(1, 8), (40, 8), (150, 4)])
def test_one_large_value(fmt, dtype, q_len, heads):
    """Values of 0.01 and one row that reaches 85, late in the sequence."""
    n = 700
    v = rows(n, 2, 128, torch.full((n,), 0.01), 2)
    v[500, :, 7] = 85.0
    run(queries(q_len, heads, 128, dtype), rows(n, 2, 128, torch.ones(n), 1), v, fmt)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("q_len", [1, 40, 150])
@pytest.mark.parametrize("large", [1e4, 1e-4])
def test_rows_that_have_left_the_window(fmt, dtype, q_len, large):
    """Rows of another size share tiles, and groups of neighbours, with rows that only some of the queries still see."""
    n = 500
    sizes = torch.ones(n)
    sizes[:n - q_len - 37] = large
    run(queries(q_len, 8, 128, dtype), rows(n, 2, 128, torch.ones(n), 1), rows(n, 2, 128, sizes, 2), fmt, 64, window=90)
    run(queries(q_len, 8, 128, dtype), rows(n, 2, 128, sizes, 1), rows(n, 2, 128, torch.ones(n), 2), fmt, 64, window=90)


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("q_len", [1, 24])
def test_results_do_not_depend_on_the_split(fmt, q_len):
    """The same long sequence alone (its keys in parts) and among others: the same rows within the bound."""
    n, kv, heads = 6000, 1, 8
    sizes = torch.ones(n)
    sizes[128:3000] = 2000.0
    sizes[3000:] = 0.01
    run(queries(q_len, heads, 128, "bf16"), rows(n, kv, 128, torch.ones(n), 1), rows(n, kv, 128, sizes, 2), fmt, 128)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("size", [1e-3, 1e-6, 1e-12, 1e4])
@pytest.mark.parametrize("zeros", ["one", "first tile", "every third", "from the middle"])
def test_rows_of_zeros(fmt, dtype, dim, shape, size, zeros):
    """A row of zeros (stored with the scale 1) counts in the sum of the weights and in nothing else."""
    q_len, n, heads, kv = shape
    sizes = torch.full((n,), size)
    at = {"one": slice(5, 6), "first tile": slice(0, 128), "every third": slice(1, n, 3), "from the middle": slice(n // 2, n)}
    sizes[at[zeros]] = 0.0
    # queries that give keys of any size scores of about one
    q = queries(q_len, heads, dim, dtype, min(1e4, 1.0 / size))
    run(q, rows(n, kv, dim, sizes, 1), rows(n, kv, dim, torch.ones(n) * size, 2), fmt)
    run(queries(q_len, heads, dim, dtype), rows(n, kv, dim, torch.ones(n), 1), rows(n, kv, dim, sizes, 2), fmt)


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("q_len", [1, 4, 40, 150])
def test_scales_of_one_that_are_not_zeros(fmt, q_len):
    """Rows whose scale is exactly 1 are rows like others."""
    n, kv, dim = 500, 2, 128
    k, v = rows(n, kv, dim, torch.ones(n), 1), rows(n, kv, dim, torch.ones(n), 2)
    # x = H e_i 8 / dim * top has one entry of top in the rotated basis: scale 1 (from rounding 1 - 2^-24 up), one code that is not zero
    top = A.TOP[fmt]
    h = torch.tensor(A.hadamard(dim)) * (8.0 / dim) * top
    for i in range(0, n, 3):
        v[i, :] = h[(i * 7) % dim].to(torch.bfloat16)
    _, scales = A.quantise(v.float().numpy(), fmt)
    assert (scales[::3] == 1.0).all()
    run(queries(q_len, 8, dim, "bf16"), k, v, fmt)


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("q_len", [1, 40, 150])
@pytest.mark.parametrize("q_by,k_by", [(1e-22, 1e-22), (1e-30, 1e-12), (1e-12, 1e-28)])
def test_scores_below_the_range(fmt, q_len, q_by, k_by):
    """Products too small for fp32 are scores of zero, and what a mask hides stays hidden."""
    n = 300
    run(queries(q_len, 8, 128, "bf16", q_by), rows(n, 2, 128, torch.ones(n) * k_by, 1), rows(n, 2, 128, torch.ones(n), 2), fmt)
    run(queries(q_len, 8, 128, "bf16", q_by), rows(n, 2, 128, torch.ones(n) * k_by, 1), rows(n, 2, 128, torch.ones(n), 2), fmt,
        window=70)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("int8", "f16"), ("int4", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_len,heads,kv", [(1, 8, 2), (1, 16, 1), (3, 8, 2), (2, 6, 2), (30, 8, 2)])
def test_query_rows_do_not_depend_on_each_other(fmt, dtype, dim, q_len, heads, kv):
    """Heads and tokens of very different sizes in one call, one of them not finite: every row as if it were alone."""
    n = 700
    k, v = rows(n, kv, dim, torch.ones(n), 1), rows(n, kv, dim, torch.ones(n), 2)
    q = queries(q_len, heads, dim, dtype)
    # sizes a factor of 2^9 apart (of fp16 down to its smallest normal numbers), large ones beside small ones
    by = 2.0 ** torch.tensor([0.0, 9.0, -9.0, 4.0])[torch.arange(q_len * heads) % 4].view(q_len, heads, 1)
    q = (q.float() * by).to(q.dtype)
    run(q, k, v, fmt)
    pages = (n + 31) // 32
    cache = E.KVCache.empty(pages, 32, kv, dim, fmt)
    E.kv_write(cache, k.to(DEV), v.to(DEV), torch.arange(n, device=DEV))
    args = (cache, torch.arange(pages, dtype=torch.int32, device=DEV)[None], cu([q_len]),
            torch.tensor([n], dtype=torch.int32, device=DEV), q_len, n)
    want = E.attention_paged(q.to(DEV), *args)
    other = q.clone()
    other[:, 1] = float("inf")
    other[:, 2] *= 8.0
    got = E.attention_paged(other.to(DEV), *args)
    keep = [h for h in range(heads) if h not in (1, 2)]
    assert torch.equal(got[:, keep], want[:, keep])
    assert torch.isnan(got[:, 1]).all() and torch.isfinite(got[:, 2]).all()


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("q_len", [1, 40, 150])
@pytest.mark.parametrize("size", [1e-27, 1e-28, 4e-29])
def test_smallest_scales(fmt, q_len, size):
    """Rows down to the format's least scale, 2^-100, keep every bit of it."""
    n = 300
    small = rows(n, 2, 128, torch.full((n,), size), 2)
    run(queries(q_len, 8, 128, "bf16"), rows(n, 2, 128, torch.ones(n), 1), small, fmt)
    run(queries(q_len, 8, 128, "bf16", 0.3 / size), small, rows(n, 2, 128, torch.ones(n), 1), fmt)
