"""Outputs that the caller gives: the queries themselves, views beside them, and overlaps that are refused."""
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from test_gpu_attention import DEV, DT, cu, make_cache

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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,kv", [(128, 8, 2), (64, 12, 4), (128, 5, 1)])
def test_prompt_over_its_queries(dtype, dim, heads, kv):
    """The output in q's place, in a fused buffer: many items, whose copies of q reach into tokens that others write."""
    lens = [300, 1, 77, 130, 64, 513, 2, 129] * 6
    x, q, k, v = fused(sum(lens), heads, kv, dim, dtype)
    want = E.attention_prompt(q, k, v, cu(lens), max(lens))
    assert torch.isfinite(want).all()
    for _ in range(20):
        y = x.clone()
        q2, k2, v2 = y[:, :heads], y[:, heads:heads + kv], y[:, heads + kv:]
        got = E.attention_prompt(q2, k2, v2, cu(lens), max(lens), out=q2)
        assert got.data_ptr() == y.data_ptr() and torch.equal(got, want)
        assert torch.equal(y[:, heads:], x[:, heads:])
    assert E.device_status() == 0


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("q_lens,kv_lens", [([1] * 24, [1 + 97 * i for i in range(24)]), ([4, 1, 3], [2777, 2, 130]),
                                            ([200, 1, 65, 130, 3, 40] * 4, [200, 300, 65, 700, 1, 500] * 4), ([40], [5000])])
def test_paged_over_its_queries(fmt, dtype, q_lens, kv_lens):
    """The same over the cache: single tokens, drafts, chunks, split keys."""
    heads, kv, dim = 8, 2, 128
    cache, table, _ = make_cache(kv_lens, kv, dim, 32, fmt, 7)
    x, q, _, _ = fused(sum(q_lens), heads, kv, dim, dtype)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    args = (cache, table, cu(q_lens), lens, max(q_lens), max(kv_lens))
    want = E.attention_paged(q, *args)
    assert torch.isfinite(want).all()
    for _ in range(20):
        y = x.clone()
        got = E.attention_paged(y[:, :heads], *args, out=y[:, :heads])
        assert torch.equal(got, want) and torch.equal(y[:, heads:], x[:, heads:])
    assert E.device_status() == 0
