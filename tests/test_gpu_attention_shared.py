"""Attention behind shared prefixes against the FP64 oracle, row by row in norm (attention_norms: close enough to see a
lost tile of keys or a part counted twice)."""
import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from attention_norms import assert_rows, bound
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
SHARE = E.SHARE_ALWAYS
FORMATS = [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int8", "f16"), ("int4", "bf16"), ("int4", "f16")]


def f64(t):
    return t.double().cpu().numpy()


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def cu(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]))


def make(lens, prefix, lead, kv, dim, page, fmt, seed):
    """A cache in which sequence b's first prefix[b] rows are those of sequence lead[b]: on the same pages as far as whole
    pages go, copies in a page of its own from there.  Rows of no sequence hold NaN."""
    g = torch.Generator().manual_seed(seed)
    dt = torch.float16 if fmt == "f16" else torch.bfloat16
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g).tolist()
    table = np.full((len(lens), max(need + [1]) + 2), -7, dtype=np.int32)
    cache = E.KVCache.empty(pages, page, kv, dim, fmt)
    if fmt in A.TOP:
        cache.k.fill_(0xFF), cache.v.fill_(0xFF), cache.k_scale.fill_(float("nan")), cache.v_scale.fill_(float("nan"))
    else:
        cache.k.fill_(float("nan")), cache.v.fill_(float("inf"))
    rows, raw = [], []
    for b, n in enumerate(lens):
        own = lead[b] == b
        keep = 0 if own else min(prefix[b], n, lens[lead[b]])
        k, v = (torch.randn((n, kv, dim), generator=g).to(dt) for _ in range(2))
        k[..., 5 % dim] *= 6.0
        if keep:
            k[:keep], v[:keep] = raw[lead[b]][0][:keep], raw[lead[b]][1][:keep]
        raw.append((k, v))
        table[b, :keep // page] = table[lead[b], :keep // page]
        for j in range(keep // page, need[b]):
            table[b, j] = order.pop()
        table[b, need[b]:] = order[-1]
        i = torch.arange(keep // page * page, n)
        if i.numel():
            slots = torch.tensor(table[b].astype(np.int64))[i // page] * page + i % page
            E.kv_write(cache, k[i].to(DEV), v[i].to(DEV), slots.to(DEV))
        if fmt in A.TOP:
            rows.append(tuple(A.read_back(*A.quantise(t.float().numpy(), fmt)) for t in (k, v)))
        else:
            rows.append((k.double().numpy(), v.double().numpy()))
    return cache, torch.tensor(table, device=DEV), rows


def shared(sizes, prefixes, q_lens, lens, heads, kv, dim, page, fmt, dtype, skip=0, max_prefix=None, seed=1, sharp=1.0, scale=None):
    """sizes: sequences of each group, from sequence ``skip`` on."""
    prefix, lead = [0] * len(lens), list(range(len(lens)))
    at = skip
    for n, p in zip(sizes, prefixes):
        ask = [b for b in range(at, at + n) if q_lens[b]] or [at]
        for b in range(at, at + n):
            prefix[b], lead[b] = p, ask[0]
        at += n
    # leads come first: a group's earlier sequences without queries get rows of their own
    for b in range(len(lens)):
        if lead[b] > b:
            prefix[b], lead[b] = 0, b
    cache, table, rows = make(lens, prefix, lead, kv, dim, page, fmt, seed)
    g = torch.Generator().manual_seed(seed + 100)
    total = sum(q_lens)
    wide = (torch.randn((total, heads * dim + 16), generator=g) * sharp).to(DT[dtype]).to(DEV)
    q = wide[:, :heads * dim].view(total, heads, dim)
    out = torch.full((total + 2, heads, dim), 3.0, dtype=DT[dtype], device=DEV)
    groups = i32(skip + np.concatenate([[0], np.cumsum(sizes)]))
    max_prefix = SHARE if max_prefix is None else max_prefix
    args = (q, cache, table, cu(q_lens), i32(lens), groups, i32(prefixes), max(q_lens), max(lens), max_prefix)
    got = E.attention_shared(*args, scale=scale, out=out[:total])
    torch.cuda.synchronize()
    assert E.device_status() == 0
    assert bool((out[total:] == 3.0).all())
    at, bounds = 0, shared.bounds
    bounds.clear()
    for b, (n, m, (k, v)) in enumerate(zip(q_lens, lens, rows)):
        want, tol = bound(f64(q[at:at + n]), k, v, 0, scale, dtype, fmt)
        bounds.append((want, tol))
        assert_rows(f64(got[at:at + n]), want, tol, f"sequence {b}: {n} queries over {m} keys")
        at += n
    assert torch.equal(E.attention_shared(*args, scale=scale), got)
    return args, got


shared.bounds = []  # of each sequence of the last call


TOKENS = [
    ([2], [256], [1, 1], [257, 300], 1, 1, 16),
    ([3], [700], [1, 1, 1], [701, 717, 830], 16, 4, 16),
    ([2], [384], [1, 1], [384, 384], 4, 2, 32),                     # the whole of both is shared
    ([40], [1000], [1] * 40, [1001 + 7 * i for i in range(40)], 6, 2, 64),
    ([3, 2], [513, 2000], [4, 1, 3, 2, 2], [520, 700, 516, 2100, 2002], 4, 1, 256),
    ([2, 3], [300, 900], [1] * 7, [900, 400, 1000, 905, 2000, 33, 0], 8, 8, 128),  # two alone behind the groups
    ([5], [1500], [0, 1, 0, 2, 1], [9, 1600, 1500, 1504, 1501], 8, 8, 16),  # sequences without queries, the first too
    ([1, 2], [5000, 640], [1, 1, 1], [5100, 650, 4000], 16, 1, 64),          # a group of one; long own keys
    ([4], [3000], [1, 1, 1, 1], [700, 3100, 1, 0], 4, 4, 32),        # a prefix longer than some lengths: not all of it, or none
    ([4], [3000], [2, 1, 3, 1], [701, 3100, 900, 3001], 4, 4, 32),
]


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sizes,prefixes,q_lens,lens,heads,kv,page", TOKENS)
def test_tokens(fmt, dtype, dim, sizes, prefixes, q_lens, lens, heads, kv, page):
    shared(sizes, prefixes, q_lens, lens, heads, kv, dim, page, fmt, dtype)


CHUNKS = [
    ([2], [256], [17, 30], [273, 400], 1, 1, 16),
    ([2], [512], [40, 33], [520, 513], 12, 2, 16),                   # chunks that begin inside the prefix
    ([3], [1300], [129, 1, 64], [1429, 1400, 1365], 3, 1, 128),
    ([2, 2], [900, 2500], [300, 20, 1, 70], [1300, 921, 2600, 2570], 8, 8, 256),
    ([2], [4000], [20, 21], [4020, 9000], 8, 1, 32),                 # few rows: keys over many CTAs
    ([3], [600], [0, 20, 30], [50, 640, 700], 16, 2, 16),
    ([2], [640], [200, 150], [700, 660], 128, 1, 64),                # every row tile is one token
]


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sizes,prefixes,q_lens,lens,heads,kv,page", CHUNKS)
def test_chunks(fmt, dtype, dim, sizes, prefixes, q_lens, lens, heads, kv, page):
    shared(sizes, prefixes, q_lens, lens, heads, kv, dim, page, fmt, dtype)


@pytest.mark.parametrize("q_len", [1, 25])
def test_sequences_before_the_groups(q_len):
    shared([2, 2], [400, 300], [q_len] * 6, [450, 500, 430, 440, 340, 500], 8, 2, 128, 16, "bf16", "bf16", skip=2)


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("max_prefix", [0, 255, 700, 100000, 2**31 - 1])
def test_the_hint_changes_no_more_than_the_order(q_len, max_prefix):
    shared([3], [900], [q_len] * 3, [980, 1000, 941], 8, 2, 128, 64, "int8", "bf16", max_prefix=max_prefix)


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("int8", "bf16"), ("int4", "f16")])
@pytest.mark.parametrize("q_len", [1, 30])
def test_sharp_scores(fmt, dtype, q_len):
    """Scores in the hundreds: one part's maximum far above the other's."""
    shared([3], [1000], [q_len] * 3, [1100, 1050, 1400], 8, 2, 128, 32, fmt, dtype, sharp=10.0, scale=0.11)


def test_many_groups_and_items():
    n = 70
    shared([2] * n, [256 + 13 * i for i in range(n)], [1] * (2 * n), [260 + 13 * (i // 2) + 90 * (i % 2) for i in range(2 * n)],
           16, 8, 128, 16, "bf16", "bf16")
    shared([2] * 20, [256 + 50 * i for i in range(20)], [33] * 40, [300 + 50 * (i // 2) + 90 * (i % 2) for i in range(40)],
           8, 4, 64, 16, "int8", "bf16")


def test_no_group_is_the_paged_call():
    args, got = shared([2], [500], [1, 1], [600, 555], 8, 2, 128, 16, "bf16", "bf16")
    q, cache, table, cq, lens, _, _, mq, mk, _ = args
    want = E.attention_paged(q, cache, table, cq, lens, mq, mk)
    none = E.attention_shared(q, cache, table, cq, lens, i32([0]), i32([]), mq, mk, SHARE)
    assert torch.equal(none, want)
    few = E.attention_shared(q, cache, table, cq, lens, i32([0, 2]), i32([500]), mq, mk, 500)
    assert torch.equal(few, want)
    one = E.attention_shared(q, cache, table, cq, lens, i32([0, 1, 2]), i32([500, 500]), mq, mk, SHARE)
    assert_rows(f64(one), f64(want), 2.0**-7 * np.linalg.norm(f64(want), axis=-1) + 1e-30)


@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_in_place_and_a_workspace_of_its_own(fmt, q_len):
    args, got = shared([4], [600], [q_len] * 4, [700, 650, 900, 640], 8, 2, 128, 16, fmt, "bf16")
    q = args[0]
    need = E.attention_shared_workspace_bytes(q.shape[0], 4, 1, 8, q.dtype, args[1], *args[-3:])
    work = torch.full((need,), 0x7F, dtype=torch.uint8, device=DEV)
    mine = q.clone()
    out = E.attention_shared(mine, *args[1:], out=mine, workspace=work)
    assert out is mine and torch.equal(mine, got)
    with pytest.raises(E.Exl3Error):
        E.attention_shared(q, *args[1:], workspace=work[:need - 16])
    assert E.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 20])
def test_pages_outside_the_cache_count_as_zeros(q_len):
    """An entry of the lead's table, and one of an own key's page, that name no page: no fault, no other sequence changed."""
    args, got = shared([2], [600], [q_len] * 3, [700, 650, 300], 8, 2, 128, 16, "int8", "bf16")
    for row, col in ((0, 3), (1, 39)):
        table = args[2].clone()
        table[row, col] = 10**6
        out = E.attention_shared(*args[:2], table, *args[3:])
        assert torch.isfinite(out).all()
        assert torch.equal(out[2 * q_len:], got[2 * q_len:])
    assert E.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 20])
def test_a_sequence_that_is_not_finite_stays_its_own(q_len):
    args, got = shared([3], [512], [q_len] * 3, [700, 650, 600], 8, 2, 128, 16, "bf16", "bf16")
    cache = args[1]
    page = int(args[2][1, 600 // 16])
    cache.k[page].fill_(float("nan"))
    out = E.attention_shared(*args)
    assert torch.equal(out[:q_len], got[:q_len]) and torch.equal(out[2 * q_len:], got[2 * q_len:])
    assert torch.isnan(out[q_len:2 * q_len]).any()


@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("groups", [[0, 9], [-3, 4], [2, 100, 2**31 - 1], [3, 1, 4], [0, 4, 0, 4, 0, 4, 1, 4, 2, 4, 0, 4] * 30])
def test_groups_that_cannot_be(groups, q_len):
    """Entries outside the batch are taken as its ends; falling ones give empty groups, or groups that overlap, whose
    results are undefined: nothing outside the tensors is touched, and the sequence of no group stays within its bound (the
    sums of its keys may be cut elsewhere)."""
    args, got = shared([4], [600], [q_len] * 5, [700, 650, 900, 640, 300], 8, 2, 128, 16, "bf16", "bf16")
    out = torch.full((5 * q_len + 3, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    prefix = i32([600] * (len(groups) - 1))
    E.attention_shared(*args[:5], i32(groups), prefix, *args[7:], out=out[:5 * q_len])
    torch.cuda.synchronize()
    assert E.device_status() == 0 and bool((out[5 * q_len:] == 3.0).all())
    if max(groups) <= 4:
        assert_rows(f64(out[4 * q_len:5 * q_len]), *shared.bounds[4])


def test_two_captured_steps():
    """Two graphs with a workspace each, replayed in turn as the lengths grow over the prefix's end."""
    args, _ = shared([4], [600], [1] * 4, [601, 602, 640, 900], 8, 2, 128, 16, "bf16", "bf16")
    q, lens = args[0], args[4]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            mine = q.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                out = E.attention_shared(mine, *args[1:])
            graphs.append((graph, mine, out))
        for step in range(4):
            graph, mine, out = graphs[step % 2]
            mine.copy_(q * (step + 1))
            lens -= 1 + step
            graph.replay()
            want = E.attention_shared(q * (step + 1), *args[1:])
            assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert E.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 20])
def test_two_calls_at_once(q_len):
    """On two streams, each with a workspace of its own: what either gives alone."""
    calls = [shared([8], [2000], [q_len] * 8, [2100 + 50 * i for i in range(8)], 8, 2, 128, 16, fmt, "bf16", seed=i)
             for i, fmt in enumerate(("bf16", "int8"))]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for (args, _), stream, mine in zip(calls, streams, outs):
            with torch.cuda.stream(stream):
                mine.append(E.attention_shared(*args))
    torch.cuda.synchronize()
    assert E.device_status() == 0
    for (_, got), mine in zip(calls, outs):
        assert all(torch.equal(o, got) for o in mine)


def test_long_lengths():
    """Offsets in the cache that pass 32 bits: pages near the end of a cache of more than 2^32 bytes a side."""
    page, kv, dim, pages = 64, 8, 128, 40000  # 2^32 bytes are 32768 pages
    cache = E.KVCache(torch.empty((pages, kv, page, dim), dtype=torch.bfloat16, device=DEV),
                      torch.empty((pages, kv, page, dim), dtype=torch.bfloat16, device=DEV), None, None, "bf16")
    lens, prefix = [700, 650, 900], 600
    g = torch.Generator().manual_seed(4)
    table = torch.arange(pages - 60, pages, dtype=torch.int32, device=DEV).view(3, 20)
    table[1:, :prefix // page] = table[0, :prefix // page]
    rows = []
    for b, n in enumerate(lens):
        k, v = (torch.randn((n, kv, dim), generator=g).to(torch.bfloat16) for _ in range(2))
        if b:
            k[:prefix], v[:prefix] = rows[0][0][:prefix], rows[0][1][:prefix]
        rows.append((k, v))
        i = torch.arange(n, device=DEV)
        E.kv_write(cache, k.to(DEV), v.to(DEV), table[b, i // page].long() * page + i % page)
    for q_len in (1, 20):
        q = torch.randn((3 * q_len, 16, dim), generator=g).to(torch.bfloat16).to(DEV)
        out = E.attention_shared(q, cache, table, cu([q_len] * 3), i32(lens), i32([0, 3]), i32([prefix]), q_len, 900, SHARE)
        for b in range(3):
            want, tol = bound(f64(q[b * q_len:(b + 1) * q_len]), *(t.double().numpy() for t in rows[b]), 0, None, "bf16", "bf16")
            assert_rows(f64(out[b * q_len:(b + 1) * q_len]), want, tol)
    assert E.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 20])
@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_rows_of_no_sequence_keep_their_output(fmt, q_len):
    """A captured step's padding behind the last sequence, and rows before the first: as they were."""
    args, got = shared([3], [600], [q_len] * 3, [700, 650, 900], 8, 2, 128, 16, fmt, "bf16")
    n = 3 * q_len
    q = torch.full((n + 7, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    q[2:n + 2] = args[0]
    out = torch.full_like(q, 5.0)
    E.attention_shared(q, *args[1:3], args[3] + 2, *args[4:], out=out)
    assert torch.equal(out[2:n + 2], got)
    assert bool((out[:2] == 5.0).all()) and bool((out[n + 2:] == 5.0).all())
    assert E.device_status() == 0
