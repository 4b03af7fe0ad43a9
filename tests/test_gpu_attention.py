"""Prompt and paged attention against the FP64 oracle, within the bound of attention_check."""
import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from attention_check import assert_close, bound
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.double().cpu().numpy()


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def prompt(lens, heads, kv, dim, dtype, window=0, scale=None, seed=1, sharp=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens)
    x = torch.randn((total, (heads + 2 * kv) * dim + pad), generator=g)
    x[:, :heads * dim] *= sharp
    x = x.to(DT[dtype]).to(DEV)
    rows = x[:, :(heads + 2 * kv) * dim].view(total, heads + 2 * kv, dim)
    q, k, v = rows[:, :heads], rows[:, heads:heads + kv], rows[:, heads + kv:]
    got = E.attention_prompt(q, k, v, cu(lens), max(lens), scale=scale, window=window)
    torch.cuda.synchronize()
    assert E.device_status() == 0
    at = 0
    for n in lens:
        want, tol = bound(f64(q[at:at + n]), f64(k[at:at + n]), f64(v[at:at + n]), window, scale, dtype, dtype)
        assert_close(f64(got[at:at + n]), want, tol, f"sequence of {n}")
        at += n
    return q, k, v, got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,heads,kv", [
    ([1], 1, 1), ([2, 1, 3], 4, 2), ([127, 128, 129], 2, 2), ([255, 1, 257], 2, 1), ([16, 17, 300], 5, 1),
    ([700], 3, 3), ([90, 0, 33], 12, 1), ([520, 40], 8, 2), ([130], 128, 1),
])
def test_prompt(dtype, dim, lens, heads, kv):
    prompt(lens, heads, kv, dim, dtype)


@pytest.mark.parametrize("dim,heads,kv", [(128, 8, 8), (64, 12, 2)])
def test_prompt_many_items(dim, heads, kv):
    """Several row tiles for every SM, of all kinds: whole, half filled, single rows."""
    prompt([300, 1, 77, 130, 64, 513, 2, 129] * 8, heads, kv, dim, "bf16")


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("int8", "bf16"), ("int4", "f16")])
def test_paged_many_items(fmt, dtype):
    q_lens = [200, 1, 65, 130, 3, 40] * 8
    kv_lens = [200, 300, 65, 700, 1, 500] * 8
    paged(q_lens, kv_lens, 16, 8, 128, 32, fmt, dtype)
    paged(q_lens, kv_lens, 16, 8, 64, 16, fmt, dtype, window=90)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 300, 5000])
@pytest.mark.parametrize("heads,kv", [(2, 2), (7, 1)])
def test_prompt_window(window, heads, kv):
    prompt([600, 5, 131], heads, kv, 128, "bf16", window=window)


def test_prompt_sharp_scores_and_strides():
    """Scores in the hundreds (the running maximum moves), a row stride wider than the heads, an own scale."""
    prompt([385, 64], 4, 2, 128, "bf16", sharp=12.0, pad=24)
    prompt([385, 64], 4, 2, 64, "f16", scale=1.7, pad=8)
    # scores that rise along the keys: every tile raises the maximum
    n, d = 900, 128
    q = torch.ones((n, 1, d), device=DEV, dtype=torch.bfloat16)
    k = (torch.arange(n, device=DEV)[:, None, None] / 16.0).expand(n, 1, d).to(torch.bfloat16).contiguous()
    v = torch.randn((n, 1, d), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    got = E.attention_prompt(q, k, v, cu([n]), n)
    want, tol = bound(f64(q), f64(k), f64(v), 0, None, "bf16", "bf16")
    assert_close(f64(got), want, tol)


def test_prompt_neighbours_do_not_leak():
    """What the next sequence holds, NaN and infinity too, does not reach the one before; nor do tokens of no sequence
    change."""
    lens, h, kv, d = [70, 61, 200], 4, 2, 128
    q, k, v, got = prompt(lens, h, kv, d, "bf16", seed=3)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    for t in (k2, v2):
        t[70:131] = float("nan")
        t[71] = float("inf")
    out = torch.full_like(got, 7.0)
    E.attention_prompt(q2, k2, v2, cu(lens), 200, out=out)
    assert torch.equal(out[:70], got[:70]) and torch.equal(out[131:], got[131:])
    assert torch.isnan(out[70:131]).any(-1).all()
    # the last 200 tokens belong to no sequence
    out = torch.full_like(got, 7.0)
    E.attention_prompt(q, k, v, cu(lens[:2]), 70, out=out)
    assert torch.equal(out[:131], got[:131]) and bool((out[131:] == 7.0).all())
    assert E.device_status() == 0


def make_cache(kv_lens, kv, dim, page, fmt, seed, spare=3, soil=True):
    """A cache whose sequences lie on shuffled pages; rows that belong to no sequence hold NaN (soil)."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in kv_lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).tolist()
    width = max(need + [1]) + 2
    table = np.full((len(kv_lens), width), -7, dtype=np.int32)
    cache = E.KVCache.empty(pages, page, kv, dim, fmt)
    if soil:
        if fmt in A.TOP:
            cache.k.fill_(0xFF), cache.v.fill_(0xFF), cache.k_scale.fill_(float("nan")), cache.v_scale.fill_(float("nan"))
        else:
            cache.k.fill_(float("nan")), cache.v.fill_(float("inf"))
    at, rows = 0, []
    for b, n in enumerate(kv_lens):
        table[b, :need[b]] = order[at:at + need[b]]
        # entries past the length name real pages of other sequences
        table[b, need[b]:] = order[-1]
        at += need[b]
        dt = torch.bfloat16 if fmt != "f16" else torch.float16
        k = torch.randn((n, kv, dim), generator=g).to(dt)
        v = torch.randn((n, kv, dim), generator=g).to(dt)
        k[..., 5 % dim] *= 6.0
        i = torch.arange(n)
        slots = torch.tensor(table[b].astype(np.int64))[i // page] * page + i % page if n else torch.empty(0, dtype=torch.int64)
        if n:
            E.kv_write(cache, k.to(DEV), v.to(DEV), slots.to(DEV))
        if fmt in A.TOP:
            rows.append(tuple(A.read_back(*A.quantise(t.float().numpy(), fmt)) for t in (k, v)))
        else:
            rows.append((k.double().numpy(), v.double().numpy()))
    return cache, torch.tensor(table, device=DEV), rows


def paged(q_lens, kv_lens, heads, kv, dim, page, fmt, dtype, window=0, seed=1, sharp=1.0, scale=None):
    cache, table, rows = make_cache(kv_lens, kv, dim, page, fmt, seed)
    g = torch.Generator().manual_seed(seed + 100)
    total = sum(q_lens)
    wide = (torch.randn((total, heads * dim + 16), generator=g) * sharp).to(DT[dtype]).to(DEV)
    q = wide[:, :heads * dim].view(total, heads, dim)
    out = torch.full((total + 2, heads, dim), 3.0, dtype=DT[dtype], device=DEV)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    args = (q, cache, table, cu(q_lens), lens, max(q_lens), max(kv_lens))
    got = E.attention_paged(*args, window=window, scale=scale, out=out[:total])
    torch.cuda.synchronize()
    assert E.device_status() == 0
    assert bool((out[total:] == 3.0).all())
    at = 0
    for n, m, (k, v) in zip(q_lens, kv_lens, rows):
        want, tol = bound(f64(q[at:at + n]), k, v, window, scale, dtype, fmt)
        assert_close(f64(got[at:at + n]), want, tol, f"{n} queries over {m} keys")
        at += n
    again = E.attention_paged(*args, window=window, scale=scale)
    assert torch.equal(again, got)
    return got


FORMATS = [("bf16", "bf16"), ("f16", "f16"), ("int8", "bf16"), ("int8", "f16"), ("int4", "bf16"), ("int4", "f16")]


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv,page", [
    ([1], [1], 1, 1, 16),
    ([1, 1, 1], [15, 0, 16], 8, 2, 16),
    ([1, 1, 1, 1], [17, 63, 64, 65], 4, 4, 32),
    ([1, 1], [1000, 33], 16, 1, 64),
    ([4, 1, 3], [777, 2, 130], 4, 1, 256),      # drafted tokens; more queries than keys
    ([3], [2], 5, 1, 16),                        # a query before the first key
    ([1] * 40, [7 * i for i in range(40)], 6, 2, 16),
    ([0, 2, 0], [50, 300, 9], 8, 8, 128),
])
def test_paged_tokens(fmt, dtype, dim, q_lens, kv_lens, heads, kv, page):
    paged(q_lens, kv_lens, heads, kv, dim, page, fmt, dtype)


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv,page", [
    ([17], [17], 1, 1, 16),
    ([33, 1, 2], [33, 500, 1], 12, 2, 16),       # a prompt, a token, more queries than keys
    ([128], [700], 2, 1, 64),
    ([129, 64], [1300, 65], 3, 1, 128),
    ([300], [301], 8, 8, 256),
    ([40], [5000], 8, 1, 32),                    # few rows: the keys are split over CTAs
    ([0, 20, 0], [50, 20, 9], 16, 2, 16),
])
def test_paged_chunks(fmt, dtype, dim, q_lens, kv_lens, heads, kv, page):
    paged(q_lens, kv_lens, heads, kv, dim, page, fmt, dtype)


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("int8", "f16"), ("int4", "bf16")])
@pytest.mark.parametrize("window", [1, 15, 64, 200, 100000])
def test_paged_window(fmt, dtype, window):
    paged([1, 2, 1], [900, 64, 0], 4, 1, 128, 16, fmt, dtype, window=window)
    paged([150, 1, 33], [900, 640, 33], 4, 2, 128, 16, fmt, dtype, window=window)
    paged([150, 1], [9000, 640], 4, 2, 64, 256, fmt, dtype, window=window)


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("int8", "bf16"), ("int4", "f16")])
def test_paged_sharp_scores(fmt, dtype):
    paged([1, 1], [2000, 700], 8, 2, 128, 32, fmt, dtype, sharp=10.0)
    paged([70, 5], [2000, 700], 8, 2, 128, 32, fmt, dtype, sharp=10.0, scale=0.11)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("q_len", [1, 40])
def test_window_does_not_follow_freed_pages(fmt, q_len):
    """Pages wholly before the window may be anyone's: their entries name soiled pages or none."""
    kv_len, page, window = 500, 16, 60
    cache, table, rows = make_cache([kv_len], 2, 128, page, fmt, 5)
    q = torch.randn((q_len, 4, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    lens = torch.tensor([kv_len], dtype=torch.int32, device=DEV)
    want = E.attention_paged(q, cache, table, cu([q_len]), lens, q_len, kv_len, window=window)
    gone = (kv_len - q_len - window + 1) // page  # pages that no query sees
    for entry in (-1, 10**6, int(table[0, -1])):
        t2 = table.clone()
        t2[0, :gone] = entry
        assert torch.equal(E.attention_paged(q, cache, t2, cu([q_len]), lens, q_len, kv_len, window=window), want)
    assert E.device_status() == 0


def test_paged_equals_prompt_over_the_same_rows():
    """A whole prompt through the cache is the prompt's attention."""
    lens, h, kv, d = [300, 77], 8, 2, 128
    q, k, v, got = prompt(lens, h, kv, d, "bf16", seed=9)
    cache = E.KVCache.empty(8, 64, kv, d, "bf16")
    table = torch.tensor([[5, 0, 3, 7, 1], [2, 6, -1, -1, -1]], dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        i = torch.arange(n, device=DEV)
        E.kv_write(cache, k[at:at + n], v[at:at + n], table[b].long()[i // 64] * 64 + i % 64)
        at += n
    out = E.attention_paged(q, cache, table, cu(lens), torch.tensor(lens, dtype=torch.int32, device=DEV), 300, 300)
    at = 0
    for n in lens:
        want, tol = bound(f64(q[at:at + n]), f64(k[at:at + n]), f64(v[at:at + n]), 0, None, "bf16", "bf16")
        assert_close(f64(out[at:at + n]), want, tol)
        at += n


@pytest.mark.parametrize("q_len", [1, 30])
def test_a_row_that_is_not_finite_stays_in_its_sequence(q_len):
    """A NaN row of one sequence makes that sequence's later queries NaN and leaves the others' bytes alone."""
    for fmt in ("bf16", "int8", "int4"):
        kv_lens = [200, 90]
        cache, table, _ = make_cache(kv_lens, 2, 128, 16, fmt, 5, soil=False)
        q = torch.randn((2 * q_len, 8, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
        lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        args = (table, cu([q_len, q_len]), lens, q_len, 200)
        want = E.attention_paged(q, cache, *args)
        assert torch.isfinite(want).all()
        bad = torch.full((1, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        E.kv_write(cache, bad, bad, table[0, :1].long() * 16 + 3)
        got = E.attention_paged(q, cache, *args)
        assert torch.isnan(got[:q_len]).all()
        assert torch.equal(got[q_len:], want[q_len:])
    assert E.device_status() == 0


@pytest.mark.parametrize("q_len", [1, 20])
def test_other_stream_and_graph(q_len):
    """On a stream of its own, and replayed from a graph with new lengths."""
    kv_lens = [500, 130]
    cache, table, rows = make_cache(kv_lens, 2, 128, 32, "int8", 5)
    q = torch.randn((2 * q_len, 8, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    off = cu([q_len, q_len])
    want = E.attention_paged(q, cache, table, off, lens, q_len, 500)
    ws = torch.empty(E.attention_paged_workspace_bytes(2 * q_len, 2, 8, 2, 128, q_len, 500), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        E.attention_paged(q, cache, table, off, lens, q_len, 500, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.attention_paged(q, cache, table, off, lens, q_len, 500, out=out, workspace=ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens.copy_(torch.tensor([90, 131], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    at = 0
    for (k, v), m in zip(rows, (90, 131)):
        m = min(m, k.shape[0])
        if m == 90:
            ref, tol = bound(f64(q[at:at + q_len]), k[:m], v[:m], 0, None, "bf16", "int8")
            assert_close(f64(out[at:at + q_len]), ref, tol)
        at += q_len


def test_refusals():
    cache, table, _ = make_cache([40], 2, 128, 16, "bf16", 1)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([40], dtype=torch.int32, device=DEV)
    one = cu([1])
    E.attention_paged(q, cache, table, one, lens, 1, 40)
    with pytest.raises(E.Exl3Error):
        E.attention_paged(q.half(), cache, table, one, lens, 1, 40)  # another type than the cache's
    with pytest.raises(E.Exl3Error):
        E.attention_paged(q[:, :3], cache, table, one, lens, 1, 40)  # heads
    with pytest.raises(E.Exl3Error):
        E.attention_paged(q, cache, table, one, lens, 0, 40)
    with pytest.raises(E.Exl3Error):
        E.attention_paged(q, cache, table, one, lens, 1, 40, scale=0.0)
    with pytest.raises(E.Exl3Error):
        E.attention_paged(q, cache, table, one, lens, 1, 40, window=-1)
    with pytest.raises(E.Exl3Error) as err:
        E.attention_paged(q, cache, table, one, lens, 1, 40, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert err.value.status == 3
    with pytest.raises(ValueError):
        E.attention_paged(q, cache, table, one.long(), lens, 1, 40)
    with pytest.raises(ValueError):
        E.attention_paged(q, cache, table[:, ::2], one, lens, 1, 40)
    with pytest.raises(ValueError):
        E.attention_prompt(q, q[:, :2].float(), q[:, :2], one)
    with pytest.raises(E.Exl3Error):
        E.attention_prompt(q, q[:, :3], q[:, :3], one)
    with pytest.raises(E.Exl3Error):
        E.attention_prompt(q[..., :96], q[:, :2, :96], q[:, :2, :96], one)
    none = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=DEV)
    assert E.attention_prompt(none, none[:, :2], none[:, :2], torch.zeros(1, dtype=torch.int32, device=DEV)).shape == (0, 4, 128)
    assert E.device_status() == 0


@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("q_len", [1, 4, 150])
@pytest.mark.parametrize("q_by,k_by,v_by", [(1.0, 1.0, 1e-6), (1e5, 1e-5, 1e5), (1e-6, 1e6, 1e-12), (1.0, 1.0, 1e-24), (3e4, 1e-3, 3e4)])
def test_paged_quantised_sizes(fmt, q_len, q_by, k_by, v_by):
    """Queries, keys and values of any size, some tokens' 64 times those of others."""
    lens, heads, kv, dim, page = 333, 8, 2, 128, 32
    g = torch.Generator().manual_seed(4)
    each = 2.0 ** torch.randint(-3, 4, (lens, 1, 1), generator=g)
    k = (torch.randn((lens, kv, dim), generator=g) * k_by * each.clamp(max=1.0)).to(torch.bfloat16)
    v = (torch.randn((lens, kv, dim), generator=g) * v_by * each.flip(0)).to(torch.bfloat16)
    q = (torch.randn((q_len, heads, dim), generator=g) * q_by).to(torch.bfloat16)
    pages = (lens + page - 1) // page
    cache = E.KVCache.empty(pages, page, kv, dim, fmt)
    E.kv_write(cache, k.to(DEV), v.to(DEV), torch.arange(lens, device=DEV))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    got = E.attention_paged(q.to(DEV), cache, table, cu([q_len]), torch.tensor([lens], dtype=torch.int32, device=DEV), q_len, lens)
    torch.cuda.synchronize()
    assert E.device_status() == 0
    kk, vv = (A.read_back(*A.quantise(t.float().numpy(), fmt)) for t in (k, v))
    want, tol = bound(q.double().numpy(), kk, vv, 0, None, "bf16", fmt)
    assert_close(f64(got), want, tol, f"{q_len} tokens")


@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("q_len", [1, 40])
def test_page_outside_the_cache_counts_as_zeros(fmt, q_len):
    kv_len, page = 300, 32
    cache, table, rows = make_cache([kv_len], 2, 128, page, fmt, 15)
    q = torch.randn((q_len, 8, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    k, v = (r.copy() for r in rows[0])
    for at, entry in ((2, -1), (4, 10**6), (7, -2**31)):
        table[0, at] = entry
        k[at * page:(at + 1) * page] = 0.0
        v[at * page:(at + 1) * page] = 0.0
    lens = torch.tensor([kv_len], dtype=torch.int32, device=DEV)
    got = E.attention_paged(q.to(DEV), cache, table, cu([q_len]), lens, q_len, kv_len)
    torch.cuda.synchronize()
    assert E.device_status() == 0
    want, tol = bound(q.double().numpy(), k, v, 0, None, "bf16", fmt)
    assert_close(f64(got), want, tol, f"{q_len} tokens")
