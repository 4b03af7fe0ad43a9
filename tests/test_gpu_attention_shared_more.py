"""Attention behind shared prefixes where what is shared changes between replays, where pages are missing, and with more
sequences and groups than the first kernel keeps in shared memory."""
import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from attention_norms import assert_rows, bound
from test_gpu_attention_shared import DEV, DT, SHARE, cu, f64, i32, make, shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("q_len", [1, 20])
def test_captured_steps_whose_prefix_changes(fmt, q_len):
    """Lengths and prefixes that move over several tiles of 128 keys in both directions between replays, so that prefixes
    are shared, shared in part or not at all: each replay against the oracle."""
    heads, kv, dim, page, n = 8, 2, 128, 16, 4
    cache, table, rows = make([900] * n, [900] * n, [0] * n, kv, dim, page, fmt, 3)
    g = torch.Generator().manual_seed(9)
    q = torch.randn((n * q_len, heads, dim), generator=g).to(torch.bfloat16).to(DEV)
    lens, prefix = i32([0] * n), i32([0])
    args = (q, cache, table, cu([q_len] * n), lens, i32([0, n]), prefix, q_len, 900, SHARE)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        E.attention_shared(*args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = E.attention_shared(*args)
        for now, p in (([250, 290, 256, 300], 900), ([500, 510, 640, 520], 900), ([650, 900, 700, 800], 600), ([300] * n, 100),
                       ([130, 0, 900, 640], 640), ([900, 850, 880, 900], 900), ([257, 400, 300, 290], 256), ([385] * n, 900)):
            lens.copy_(i32(now))
            prefix.copy_(i32([p]))
            out.fill_(9.0)
            graph.replay()
            for b, m in enumerate(now):
                mine = slice(b * q_len, (b + 1) * q_len)
                want, tol = bound(f64(q[mine]), *(r[:m] for r in rows[b]), 0, None, "bf16", fmt)
                assert_rows(f64(out[mine]), want, tol, f"lengths {now}, prefix {p}, sequence {b}")
    torch.cuda.synchronize()
    assert E.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int4", "f16")])
def test_missing_pages_are_zeros(fmt, dtype, q_len):
    """A page of the shared prefix (read through the lead's table, so by both) and one of a sequence's own keys that name no
    page of the cache: the oracle's rows there are zeros; who does not read them is what it was, bit by bit."""
    page, lens, prefix = 16, [700, 650, 300], 600
    args, got = shared([2], [prefix], [q_len] * 3, lens, 8, 2, 128, page, fmt, dtype)
    cache, table, rows = make(lens, [prefix, prefix, 0], [0, 0, 2], 2, 128, page, fmt, 1)  # the same once more
    assert torch.equal(table, args[2])
    for row, col, hurt in ((0, 3, (0, 1)), (1, 39, (1,)), (0, 41, (0,)), (2, 0, (2,))):
        for entry in (10**6, -1):
            wrong = args[2].clone()
            wrong[row, col] = entry
            out = E.attention_shared(*args[:2], wrong, *args[3:])
            for b, m in enumerate(lens):
                mine = slice(b * q_len, (b + 1) * q_len)
                if b not in hurt:
                    assert torch.equal(out[mine], got[mine])
                    continue
                k, v = (r.copy() for r in rows[b])
                k[col * page:(col + 1) * page] = 0.0
                v[col * page:(col + 1) * page] = 0.0
                want, tol = bound(f64(args[0][mine]), k, v, 0, None, dtype, fmt)
                assert_rows(f64(out[mine]), want, tol, f"page {col} of {row}, sequence {b}")
    assert E.device_status() == 0


def lengths(sizes, prefixes, silent, q_len, seed):
    """(queries, lengths) of each sequence: own keys behind its group's prefix, none asked of those in ``silent``."""
    rng = np.random.default_rng(seed)
    q, lens = [], []
    for n, p in zip(sizes, prefixes):
        for _ in range(n):
            q.append(0 if len(q) in silent else q_len)
            lens.append(p + q_len + int(rng.integers(0, 90)))
    return q, lens


@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("sizes", [[1023, 1], [1024], [1000, 25], [2, 1100, 3], [2] * 255, [2] * 256, [2] * 257, [2, 1, 3] * 130,
                                   [2] * 600, [3, 2] * 300], ids=lambda s: f"{len(s)}x{s[0]}")
def test_more_than_the_first_kernel_holds(sizes, q_len):
    """Lengths of up to 1024 sequences and 256 groups are kept in shared memory: at those borders and past them."""
    n = sum(sizes)
    prefixes = [256 + 128 * (i % 3) + 5 * (i % 7) for i in range(len(sizes))]
    silent = {b for b in (0, 31, 255, 256, 511, 1023, 1024, 1025, n - 1) if b % 2}
    q, lens = lengths(sizes, prefixes, silent, q_len, 4)
    shared(sizes, prefixes, q, lens, 2, 1, 64, 16, "bf16", "bf16", seed=len(sizes))


@pytest.mark.parametrize("q_len", [1, 20])
def test_alone_before_and_behind_many_groups(q_len):
    sizes = [2] * 300
    prefixes = [256 + 3 * (i % 50) for i in range(300)]
    q, lens = lengths([5] + sizes + [700], [0] + prefixes + [10], {3, 304, 900}, q_len, 8)
    shared(sizes, prefixes, q, lens, 2, 1, 64, 16, "int8", "bf16", skip=5)


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("int8", "f16"), ("int4", "bf16")])
@pytest.mark.parametrize("sizes,prefixes,q_lens,lens,heads,kv", [
    ([2], [600], [20, 20, 20, 20], [640, 700, 9000, 300], 8, 1),     # alone and long beside a short prefix
    ([1, 2], [8000, 300], [33, 17, 40], [8100, 400, 350], 4, 2),     # a group of one: nothing is shared of its prefix
    ([3], [5000], [20, 1, 30, 64], [5020, 5100, 5030, 5200], 12, 2),
    ([2], [700], [40, 40, 0, 40], [760, 777, 8000, 40], 4, 1),       # long, without queries
])
def test_long_own_keys_in_row_tiles(fmt, dtype, sizes, prefixes, q_lens, lens, heads, kv):
    """Own keys far longer than the rest behind a prefix: parts by each sequence's own length."""
    for max_prefix in (SHARE, max(prefixes)):
        shared(sizes, prefixes, q_lens, lens, heads, kv, 128, 64, fmt, dtype, max_prefix=max_prefix)
