"""Row tiles: items of every kind one after the other in the same CTAs."""
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from test_gpu_attention import DEV, cu, make_cache, paged, prompt

pytestmark = pytest.mark.gpu

# (query tokens, keys): long chunks whose halves drift apart, then items of at most 128 rows whose halves meet in shared
# memory: of one block, of several, and without any key
MIXED = [(200, 2500), (1, 40), (3, 0), (40, 700), (2, 1), (129, 130), (1, 64)]


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("dim,heads,kv", [(128, 8, 1), (64, 8, 4)])
def test_halves_meet_after_long_items(fmt, dtype, dim, heads, kv):
    q_lens, kv_lens = zip(*(MIXED * 6))
    paged(list(q_lens), list(kv_lens), heads, kv, dim, 64, fmt, dtype)


def test_prompts_of_one_block_after_long_ones():
    prompt([700, 1, 20, 300, 64, 2] * 12, 8, 4, 128, "bf16")


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_repeats_to_the_byte(fmt):
    """Several items for every SM, two hundred times."""
    q_lens, kv_lens = (list(x) for x in zip(*(MIXED * 12)))
    kv, heads, dim = 8, 32, 128
    cache, table, _ = make_cache(kv_lens, kv, dim, 32, fmt, 3)
    q = torch.randn((sum(q_lens), heads, dim), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    args = (q, cache, table, cu(q_lens), lens, max(q_lens), max(kv_lens))
    want = E.attention_paged(*args)
    assert torch.isfinite(want).all()
    for _ in range(200):
        assert torch.equal(E.attention_paged(*args), want)
    assert E.device_status() == 0
