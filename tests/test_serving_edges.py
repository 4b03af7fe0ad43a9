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
