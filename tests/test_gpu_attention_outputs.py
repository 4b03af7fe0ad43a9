"""Outputs that the caller gives: the queries themselves, views beside them, and overlaps that are refused."""
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from test_gpu_attention import DEV, DT, cu

pytestmark = pytest.mark.gpu


def fused(tokens, heads, kv, dim, dtype="bf16", seed=3):
    x = torch.randn((tokens, heads + 2 * kv, dim), generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).to(DEV)
    return x, x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]


def test_refused_overlaps():
    heads, kv, dim, n = 8, 2, 128, 40
    x, q, k, v = fused(n, heads, kv, dim)
    phases, amp = E.rope_phases(dim)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    slots = torch.arange(n, device=DEV)
    cache = E.KVCache.empty(20, 16, kv, dim, "bf16")
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    E.kv_write(cache, k, v, slots)
    rows = cache.k.view(-1, dim)[:heads * n].view(n, heads, dim)  # the cache's own memory
    before = x.clone()
    with pytest.raises(ValueError):
        E.attention_prompt(q, k, v, cu([n]), n, out=x[:, kv:heads + kv])  # reaches into k
    with pytest.raises(ValueError):
        E.attention_prompt(q.clone(), k, v, cu([n]), n, out=x[:, 2 * kv:])
    with pytest.raises(ValueError):
        E.kv_write(cache, k, v, slots, q=q.clone(), positions=pos, phases=phases, amplitude=amp, q_out=x[:, kv:heads + kv])
    with pytest.raises(ValueError):
        E.kv_write(cache, k, v, slots, q=q, positions=pos, phases=phases, amplitude=amp, q_out=rows)
    with pytest.raises(ValueError):
        E.attention_paged(q, cache, table, cu([n]), lens, n, n, out=rows)
    out = cache.v.view(-1)[:n * kv * dim].view(n, kv, dim)
    with pytest.raises(ValueError):
        E.kv_read(cache, slots, k=out)
    with pytest.raises(ValueError):
        E.kv_read(cache, slots, v=out)
    one = torch.empty((n, kv, dim), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        E.kv_read(cache, slots, k=one, v=one)
    assert torch.equal(x, before)
    # beside its inputs in the same rows: other heads of the buffer
    wide = torch.zeros((n, 2 * heads + 2 * kv, dim), dtype=torch.bfloat16, device=DEV)
    wide[:, :heads + 2 * kv] = x
    q2, k2, v2, o2 = wide[:, :heads], wide[:, heads:heads + kv], wide[:, heads + kv:heads + 2 * kv], wide[:, heads + 2 * kv:]
    want = E.attention_prompt(q, k, v, cu([n]), n)
    assert torch.equal(E.attention_prompt(q2, k2, v2, cu([n]), n, out=o2), want)
    assert torch.equal(E.rope(q2, pos, phases, out=o2), E.rope(q, pos, phases))
    assert torch.equal(wide[:, :heads + 2 * kv], x)
    assert E.device_status() == 0
