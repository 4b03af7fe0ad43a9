"""Page tables, norms with the rotation, the cache and attention behind a shared prefix together: the example attention
layer's single-token steps (one CUDA graph, its lengths and tables moving on the GPU) agree with prompt attention over the
whole sequences, and every page comes back."""
import os
import sys

import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from test_gpu_attention_layer import STEP, UNIT

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [None, E.SHARE_ALWAYS])
@pytest.mark.parametrize("shared", [0, 320])
@pytest.mark.parametrize("fmt", ["bf16", "f16", "int8", "int4"])
def test_steps_agree_with_prompts(fmt, shared, hint):
    """Tolerance as for the layer without norms: the normed heads are the same rounded rows on both sides but for the
    projection's own roundings, which the norm scales with the row."""
    import attention_layer

    if hint is not None and not shared:
        pytest.skip("nothing to share")
    got, want, _ = attention_layer.run(fmt, steps=5, seqs=5, prompt=260, hidden=512, heads=8, kv_heads=2, shared=shared,
                                       norm=True, hint=hint)
    torch.cuda.synchronize()
    assert got.shape == want.shape == (5, 8, 128)
    got, want = got.double().cpu().numpy(), want.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off <= 6 * UNIT[fmt] + 2 * STEP[fmt] / 3


def test_refused_tokens_write_nothing():
    """A step whose pages run out: the refused sequence's rows go nowhere, the others' attention is what it is alone."""
    page, kv, dim, heads = 16, 2, 64, 4
    tables = E.KVTables.empty(3, 64, 3, page)  # three pages for three sequences
    cache = E.KVCache.empty(3, page, kv, dim, "bf16")
    g = torch.Generator().manual_seed(1)
    total = 50

    def rows(n):
        return torch.randn((total, n, dim), generator=g).to(torch.bfloat16).cuda()

    q, k, v = rows(heads), rows(kv), rows(kv)
    new = torch.tensor([20, 20, 10], dtype=torch.int32, device="cuda")  # two pages, two, one: the second is refused
    cu, positions, slots, granted = E.kv_plan(tables, new, total)
    assert granted.tolist() == [True, False, False] and tables.kv_lens.tolist() == [20, 0, 0]
    cache.k.fill_(7.0)
    E.kv_write(cache, k, v, slots)
    assert int((cache.k != 7.0).any(-1).sum()) == 20 * kv
    out = E.attention_paged(q, cache, tables.block_table, cu, tables.kv_lens, 20, 64)
    alone = E.attention_prompt(q[:20], k[:20], v[:20], torch.tensor([0, 20], dtype=torch.int32, device="cuda"), 20)
    # both bf16 results of the same rows: two roundings of the result and of the weights
    assert float((out[:20].double() - alone.double()).norm() / alone.double().norm()) <= 4 * 2.0**-8
    assert not out[20:].any()  # no key of theirs is in the cache
    E.kv_release(tables, torch.tensor([True, False, False], device="cuda"))
    _, _, slots, granted = E.kv_plan(tables, torch.tensor([0, 20, 10], dtype=torch.int32, device="cuda"), total)
    assert granted.tolist() == [True, True, True] and int(tables.free_count) == 0 and bool((slots[:30] >= 0).all())
