"""Windows of paged attention: what lies before them, and windows larger than any sequence."""
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from test_gpu_attention import DEV, DT, cu, make_cache

pytestmark = pytest.mark.gpu


def spoil(cache, slots, kv, dim):
    """Rows that are not finite (in a quantised cache: NaN scales) in the given slots."""
    dtype = torch.float16 if cache.fmt == "f16" else torch.bfloat16
    k = torch.full((len(slots), kv, dim), float("inf"), dtype=dtype, device=DEV)
    v = torch.full((len(slots), kv, dim), float("nan"), dtype=dtype, device=DEV)
    E.kv_write(cache, k, v, torch.tensor(slots, device=DEV))


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("q_len,kv_len,window", [(1, 500, 60), (40, 500, 60), (150, 700, 90), (150, 391, 129), (24, 3000, 2500),
                                                 (40, 500, 1), (40, 514, 474)])
def test_rows_before_every_window(fmt, dtype, dim, page, q_len, kv_len, window):
    """Rows that no query of the call sees any more, in pages that are still read, may hold anything."""
    cache, table, _ = make_cache([kv_len], 2, dim, page, fmt, 5)
    q = torch.randn((q_len, 16, dim), generator=torch.Generator().manual_seed(6)).to(DT[dtype]).to(DEV)
    lens = torch.tensor([kv_len], dtype=torch.int32, device=DEV)
    args = (q, cache, table, cu([q_len]), lens, q_len, kv_len)
    want = E.attention_paged(*args, window=window)
    assert torch.isfinite(want).all()
    first = kv_len - q_len - window + 1
    assert first > 0
    ids = table[0].tolist()
    spoil(cache, [ids[j // page] * page + j % page for j in range(first)], 2, dim)
    got = E.attention_paged(*args, window=window)
    torch.cuda.synchronize()
    assert E.device_status() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [70, 1]), ([40, 200], [3, 500]), ([300], [290])])
def test_a_window_of_any_size(fmt, q_lens, kv_lens):
    """Windows beyond every length, up to the largest int32, with queries before the first key among them, are none."""
    cache, table, _ = make_cache(kv_lens, 2, 128, 32, fmt, 5)
    q = torch.randn((sum(q_lens), 8, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    args = (q, cache, table, cu(q_lens), lens, max(q_lens), max(kv_lens))
    want = E.attention_paged(*args)
    for window in (2**20, 2**30 - 1, 2**30, 2**31 - 300, 2**31 - 1):
        assert torch.equal(E.attention_paged(*args, window=window), want)
    k = torch.randn((sum(q_lens), 2, 128), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(DEV)
    want = E.attention_prompt(q, k, k, cu(q_lens))
    for window in (2**20, 2**30, 2**31 - 1):
        assert torch.equal(E.attention_prompt(q, k, k, cu(q_lens), window=window), want)
    assert E.device_status() == 0
