"""The example attention layer behind a shared beginning when its sequences end one after the other: the beginning stays
for those that still read it, and comes back with the last."""
import os
import sys

import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from test_gpu_attention_layer import UNIT

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [None, E.SHARE_ALWAYS])
@pytest.mark.parametrize("order", [[0, 1, 2], [1, 0, 2], [2, 1, 0]])
def test_sequences_end_in_any_order(order, hint):
    """Steps after each end, over enough tokens that free pages are taken (the ones given back last come first): the last
    step's rows are prompt attention's over the whole sequences.  Tolerance as for the layer's other steps."""
    import attention_layer

    begin, lens, steps, hidden = 320, [60, 70, 130], 12, 512
    g = torch.Generator(device="cuda").manual_seed(7)

    def rows(n):
        return torch.randn((n, hidden), generator=g, device="cuda").to(torch.bfloat16)

    layer = attention_layer.AttentionLayer(hidden, 8, 2, 128, 3, 640, "bf16")
    t = layer.tables
    first = rows(begin)
    layer.prompt(first, [begin, 0, 0])
    layer.share(begin, hint)
    tokens = [[first, rows(n)] for n in lens]
    layer.step(torch.cat([x[-1] for x in tokens]), torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens))
    running = [0, 1, 2]
    shared = t.block_table[0, :begin // layer.page].tolist()
    for end in order:
        layer.end(torch.tensor([b == end for b in range(3)], device="cuda"))
        running.remove(end)
        free = t.free_pages[:int(t.free_count)].tolist()
        assert len(set(free)) == len(free)
        if not running:
            assert sorted(free) == list(range(layer.cache.num_pages))
            break
        for b in running:
            assert not set(free) & set(t.block_table[b, :int(t.held[b])].tolist()), f"pages of {b} are free after the end of {end}"
        held = layer.cache.k[shared].clone()
        for _ in range(steps):
            x = rows(len(running))
            for i, b in enumerate(running):
                tokens[b].append(x[i:i + 1])
            out = layer.step(x)
        assert torch.equal(layer.cache.k[shared], held)
        whole = [torch.cat(tokens[b]) for b in running]
        n = [x.shape[0] for x in whole]
        every = layer.prompt(torch.cat(whole), n, keep=False)
        want = every[torch.tensor(n, device="cuda").cumsum(0) - 1].double().cpu().numpy()
        got = out.double().cpu().numpy()
        assert np.linalg.norm(got - want) / np.linalg.norm(want) <= 6 * UNIT["bf16"]
    # the layer begins anew
    layer.prompt(rows(30), [10, 10, 10])
    layer.step(rows(3))
    assert t.kv_lens.tolist() == [11, 11, 11] and E.device_status() == 0
