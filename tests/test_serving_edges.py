"""The ends of what the calls of a serving step accept, without a GPU."""
import os
import sys

import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from exl3_trellis_quantized_gb300 import binding as B
from test_attention_abi import EINVAL, FAKE, L  # noqa: F401
from test_serving_abi import ints, on_cpu, rows, some_tables, tables  # noqa: F401


def test_stacks_stay_below_where_sums_saturate(L):  # noqa: F811
    """A sum of pages that saturates (2^30) must not look like one that the stack holds, so no stack holds 2^30."""
    full = tables(capacity=1 << 30)
    assert L.exl3_kv_plan(full, FAKE, 5, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == EINVAL
    assert L.exl3_kv_release(full, FAKE, FAKE, FAKE, FAKE, FAKE, None) == EINVAL


def test_tables_refuse_such_a_stack(on_cpu, monkeypatch):  # noqa: F811
    monkeypatch.setattr(B, "_apart", lambda *args, **others: None)  # tensors without memory all lie at 0

    def made(capacity):
        return B.KVTables(ints(3, 4, device="meta"), ints(3, device="meta"), ints(3, device="meta"),
                          ints(capacity, device="meta"), ints(1, device="meta"), 16)

    assert made((1 << 30) - 1).free_pages.numel() == (1 << 30) - 1
    with pytest.raises(ValueError, match="free_pages"):
        made(1 << 30)


def test_norm_alone_checks(on_cpu):  # noqa: F811
    """With a weight the rows need no positions; half of a rotation is refused."""
    positions, phases, w = ints(2), ints(16, dtype=torch.int64), torch.zeros(64, dtype=torch.bfloat16)
    E.rope(rows(), weight=w)
    E.rope(rows(), weight=w.expand(2, 64))
    assert on_cpu == ["exl3_norm_rope"] * 2
    on_cpu.clear()
    for bad in (dict(), dict(positions=positions), dict(phases=phases), dict(positions=positions, weight=w),
                dict(phases=phases, weight=w), dict(axes=ints(16, dtype=torch.uint8), weight=w), dict(weight=w[:32]),
                dict(weight=w.to("meta"))):
        with pytest.raises(ValueError):
            E.rope(rows(), **bad)
    assert not on_cpu


def pays(L, n, prefix, groups=1, alone=0, q=1, h=32, kv=8, fmt=1, dtype=1):  # noqa: F811
    """Whether n sequences of q tokens in so many groups, and some alone, share their prefix."""
    return L.exl3_attention_shared_pays((n + alone) * q, n + alone, n, groups, h, kv, 128, dtype, fmt, q, prefix)


def test_sharing_pays_where_it_was_measured_to(L):  # noqa: F811
    """Sizes of which both calls were timed, a tenth apart at the least, on the side that was faster (fmt 1: 16 bits, 2: 8)."""
    shared = [dict(n=16, prefix=8192), dict(n=16, prefix=8192, fmt=2), dict(n=64, prefix=512), dict(n=32, prefix=2048),
              dict(n=32, prefix=2048, fmt=2), dict(n=8, prefix=32768), dict(n=8, prefix=32768, fmt=2),
              dict(n=32, prefix=4096, groups=16), dict(n=128, prefix=4096, groups=64), dict(n=500, prefix=512, groups=250),
              dict(n=256, prefix=512, groups=64), dict(n=1000, prefix=1024, groups=250, fmt=2),
              dict(n=32, alone=32, prefix=8192), dict(n=32, alone=32, prefix=8192, fmt=2), dict(n=8, alone=56, prefix=32768),
              dict(n=8, prefix=4096, q=8), dict(n=40, prefix=1024, q=8), dict(n=40, prefix=1024, q=8, fmt=2),
              dict(n=8, prefix=8192, q=30), dict(n=16, prefix=16000, q=100), dict(n=16, prefix=8000, q=100)]
    paged = [dict(n=3, prefix=700), dict(n=2, prefix=8192), dict(n=4, prefix=8192), dict(n=8, prefix=4096), dict(n=16, prefix=2048),
             dict(n=8, prefix=8192, fmt=2), dict(n=16, prefix=4096, fmt=2), dict(n=4, prefix=16384, fmt=2),
             dict(n=4, prefix=32768, fmt=2), dict(n=32, prefix=512, fmt=2), dict(n=128, prefix=2048, groups=64, fmt=2),
             dict(n=128, prefix=4096, groups=64, fmt=2), dict(n=128, prefix=8192, groups=64, fmt=2),
             dict(n=32, prefix=8192, groups=16, fmt=2), dict(n=500, prefix=2048, groups=250, fmt=2),
             dict(n=2, alone=60, prefix=8192), dict(n=2, alone=60, prefix=8192, fmt=2), dict(n=8, alone=56, prefix=8192, fmt=2),
             dict(n=4, alone=60, prefix=32768, fmt=2), dict(n=4, prefix=4096, q=8), dict(n=16, prefix=512, q=8),
             dict(n=4, prefix=2048, q=30), dict(n=16, prefix=2048, q=30), dict(n=16, prefix=4000, q=100)]
    for args in shared:
        assert pays(L, **args) == 1, args
    for args in paged:
        assert pays(L, **args) == 0, args
    # by rule, whatever the sizes: few fp16 rows over codes, groups of one, no groups
    assert pays(L, 64, 8192, dtype=0, fmt=2) == pays(L, 64, 8192, groups=64) == pays(L, 64, 8192, groups=0) == 0
    assert pays(L, 64, 255) == pays(L, 65, 8192, alone=-1) == pays(L, -1, 8192, alone=64) == pays(L, 64, 8192, h=7) == 0


def test_more_own_keys_change_nothing(L):  # noqa: F811
    """max_kv, which a captured step fills with its capacity, takes no part in the choice."""
    def size(max_kv, max_prefix):
        return L.exl3_attention_shared_workspace_bytes(1739, 7, 1, 32, 8, 128, 1, 3, 700, max_kv, max_prefix)

    for max_kv in (17999, 18000, 18001, 40000):
        assert L.exl3_attention_paged_workspace_bytes(1739, 7, 32, 8, 128, 700, max_kv, 0) != size(max_kv, 16000) > 0


def test_sharers_steer(on_cpu, monkeypatch):  # noqa: F811
    asked, passed = [], []

    class Library:
        def __getattr__(self, name):
            return lambda *args: passed.append(args[15]) or 0

    monkeypatch.setattr(B, "lib", lambda: Library())
    monkeypatch.setattr(B, "_sharing_pays", lambda *sizes: asked.append(sizes[2]) or sizes[2] >= 2)
    cache = B.KVCache.empty(3, 16, 2, 64, "int8", device="cpu")
    args = dict(q=rows(3), cache=cache, block_table=ints(3, 3), cu_q=ints(4), kv_lens=ints(3), cu_groups=ints(2), prefix_lens=ints(1),
                max_q=1, max_kv=9, max_prefix=700)
    for sharers in (None, 3, 2, 1, 0):
        E.attention_shared(**args, sharers=sharers)
    E.attention_shared(**{**args, "max_prefix": E.SHARE_ALWAYS}, sharers=1)
    assert passed == [700, 700, 700, 0, 0, E.SHARE_ALWAYS] and asked == [3, 2, 1, 0]
    for sharers in (-1, 4):
        with pytest.raises(ValueError):
            E.attention_shared(**args, sharers=sharers)
        with pytest.raises(ValueError):
            E.attention_shared_workspace_bytes(3, 3, 1, 2, torch.bfloat16, cache, 1, 9, 700, sharers=sharers)


def example_layer(**attributes):
    """The example's layer without tensors on a GPU."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from attention_layer import AttentionLayer

    layer = object.__new__(AttentionLayer)
    layer.__dict__.update(dict(window=0, page=16, groups=None, tables=some_tables()), **attributes)
    return layer


def test_a_layer_with_a_window_shares_nothing(on_cpu):  # noqa: F811
    """Attention behind shared prefixes has no window: a layer that has one must not lose it."""
    with pytest.raises(ValueError, match="window"):
        example_layer(window=100).share(32)


def test_a_layer_shares_whole_pages(on_cpu):  # noqa: F811
    for tokens in (40, 0, -16):
        with pytest.raises(ValueError, match="pages"):
            example_layer().share(tokens)


def test_no_whole_prompts_behind_a_shared_beginning(on_cpu):  # noqa: F811
    """Prompt attention sees the new rows only."""
    with pytest.raises(ValueError, match="step"):
        example_layer(groups=ints(2)).prompt(rows(), [1, 1, 0])
