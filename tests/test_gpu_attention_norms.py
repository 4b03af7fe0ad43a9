"""Paged attention held row by row in norm (attention_norms), where the worst-case bound would let lost keys pass; and a
graph replayed with new lengths, every sequence checked."""
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from attention_norms import assert_rows, bound
from test_gpu_attention import DEV, DT, FORMATS, cu, f64, make_cache

pytestmark = pytest.mark.gpu


def check(got, q, rows, q_lens, kv_lens, dtype, fmt, window=0, scale=None):
    at = 0
    for n, m, (k, v) in zip(q_lens, kv_lens, rows):
        want, tol = bound(f64(q[at:at + n]), k[:m], v[:m], window, scale, dtype, fmt)
        assert_rows(f64(got[at:at + n]), want, tol, f"{n} queries over {m} keys")
        at += n


def paged(q_lens, kv_lens, heads, kv, dim, page, fmt, dtype, window=0, sharp=1.0, scale=None):
    cache, table, rows = make_cache(kv_lens, kv, dim, page, fmt, 21)
    g = torch.Generator().manual_seed(22)
    q = (torch.randn((sum(q_lens), heads, dim), generator=g) * sharp).to(DT[dtype]).to(DEV)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    got = E.attention_paged(q, cache, table, cu(q_lens), lens, max(q_lens), max(kv_lens), window=window, scale=scale)
    torch.cuda.synchronize()
    assert E.device_status() == 0
    check(got, q, rows, q_lens, kv_lens, dtype, fmt, window, scale)


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv,dim,page,window,sharp,scale", [
    ([1, 1], [2000, 700], 8, 2, 128, 32, 0, 10.0, None),
    ([70, 5], [2000, 700], 8, 2, 128, 32, 0, 10.0, 0.11),
    ([1] * 20, [7 + 211 * i for i in range(20)], 8, 2, 128, 64, 0, 1.0, None),  # ranges cut inside sequences
    ([4, 1, 3], [777, 2, 3130], 4, 1, 64, 256, 0, 1.0, None),
    ([40], [5000], 8, 1, 128, 32, 0, 1.0, None),        # parts of the keys
    ([40, 7], [5000, 4100], 8, 1, 64, 16, 0, 1.0, None),
    ([129, 64], [1300, 65], 3, 1, 128, 128, 0, 1.0, None),
    ([300, 1, 20], [900, 640, 20], 8, 2, 64, 32, 200, 1.0, None),
    ([300, 1, 20], [900, 640, 20], 8, 2, 128, 256, 77, 1.0, None),
    ([1, 2], [900, 640], 4, 2, 128, 16, 77, 1.0, None),
])
def test_rows(fmt, dtype, q_lens, kv_lens, heads, kv, dim, page, window, sharp, scale):
    paged(q_lens, kv_lens, heads, kv, dim, page, fmt, dtype, window, sharp, scale)


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("q_len", [1, 20])
def test_replay_with_new_lengths(fmt, dtype, q_len):
    """The graph's work follows the lengths of the replay, not those of the capture."""
    most = [500, 330, 129]
    cache, table, rows = make_cache(most, 2, 128, 32, fmt, 5)
    q = torch.randn((3 * q_len, 8, 128), generator=torch.Generator().manual_seed(6)).to(DT[dtype]).to(DEV)
    lens = torch.tensor([40, 330, 100], dtype=torch.int32, device=DEV)
    off = cu([q_len] * 3)
    out = torch.empty_like(q)
    ws = torch.empty(E.attention_paged_workspace_bytes(3 * q_len, 3, 8, 2, 128, q_len, 500), dtype=torch.uint8, device=DEV)
    E.attention_paged(q, cache, table, off, lens, q_len, 500, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.attention_paged(q, cache, table, off, lens, q_len, 500, out=out, workspace=ws)
    for now in ([500, 31, 129], [64, 65, 1], [0, 330, 128]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert E.device_status() == 0
        check(out, q, rows, [q_len] * 3, now, dtype, fmt)
