"""Page tables, norms with the rotation and attention behind shared prefixes without a GPU: refusals on the host, workspace
sizes, the binding's own checks, the oracle's norm."""
import math

import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from exl3_trellis_quantized_gb300 import binding as B
from oracle import attention_oracle as A
from test_attention_abi import (BAD_CACHES, BAD_HEADS, BAD_TURNS, BF16, EINVAL, EUNSUPPORTED, EWORKSPACE, F16, FAKE, L,  # noqa: F401
                                OK, cache, heads, turn)

MISALIGNED = (None, FAKE + 2)


def tables(table=FAKE, lens=FAKE, held=FAKE, free=FAKE, count=FAKE, batch=3, width=4, page=16, capacity=10):
    return B._Tables(table, lens, held, free, count, batch, width, page, capacity)


BAD_TABLES = [tables(table=None), tables(table=FAKE + 2), tables(lens=None), tables(lens=FAKE + 1), tables(held=None),
              tables(held=FAKE + 3), tables(free=None), tables(free=FAKE + 2), tables(count=None), tables(count=FAKE + 2),
              tables(batch=-1), tables(batch=(1 << 22) + 1), tables(width=0), tables(width=1 << 27), tables(page=8),
              tables(page=48), tables(page=512), tables(capacity=0), tables(capacity=(1 << 30) + 1)]


def test_plan_refused(L):  # noqa: F811
    def call(t=tables(), new=FAKE, total=5, lens=FAKE, held=FAKE, count=FAKE, cu=FAKE, pos=FAKE, slots=FAKE, granted=FAKE):
        return L.exl3_kv_plan(t, new, total, lens, held, count, cu, pos, slots, granted, None)

    for t in BAD_TABLES:
        assert call(t=t) == EINVAL
    for name in ("new", "lens", "held", "count", "cu", "pos"):
        for p in MISALIGNED:
            assert call(**{name: p}) == EINVAL, name
    assert call(t=None) == call(slots=None) == call(slots=FAKE + 4) == call(granted=None) == EINVAL
    assert call(total=-1) == call(total=(1 << 22) + 1) == EINVAL


def test_release_refused(L):  # noqa: F811
    def call(t=tables(), ended=FAKE, shared=FAKE, lens=FAKE, held=FAKE, count=FAKE):
        return L.exl3_kv_release(t, ended, shared, lens, held, count, None)

    for t in BAD_TABLES:
        assert call(t=t) == EINVAL
    for name in ("lens", "held", "count"):
        for p in MISALIGNED:
            assert call(**{name: p}) == EINVAL, name
    assert call(t=None) == call(ended=None) == call(shared=FAKE + 2) == EINVAL


def norm(weight=FAKE, stride=0, eps=1e-6):
    return B._Norm(weight, stride, eps)


def axes(at=FAKE, n=3):
    return B._Axes(at, n)


BAD_NORMS = [norm(None), norm(FAKE + 8), norm(stride=-8), norm(stride=4), norm(stride=(1 << 32) + 8), norm(eps=0.0),
             norm(eps=-1e-6), norm(eps=1e-40), norm(eps=math.nan), norm(eps=math.inf)]
BAD_AXES = [axes(None), axes(n=0), axes(n=256)]


def test_norm_rope_refused(L):  # noqa: F811
    def call(x=heads(), dtype=BF16, tokens=3, n=4, dim=128, w=norm(), r=turn(), ax=axes(), out=FAKE * 2, ot=1024, oh=128):
        return L.exl3_norm_rope(x, dtype, tokens, n, dim, w, r, ax, out, ot, oh, None)

    for h in BAD_HEADS:
        assert call(x=h) == EINVAL
    for r in BAD_TURNS:
        assert call(r=r) == EINVAL
    for w in BAD_NORMS:
        assert call(w=w) == EINVAL
    for ax in BAD_AXES:
        assert call(ax=ax) == EINVAL
    assert call(w=None, r=None, ax=None) == EINVAL  # nothing to do with the rows
    assert call(r=None) == EINVAL                   # axes of no rotation
    assert call(x=None) == call(out=None) == call(out=FAKE, ot=2048) == call(n=0) == call(dtype=2) == call(tokens=-1) == EINVAL
    assert call(dim=96) == EUNSUPPORTED
    assert call(tokens=0, x=heads(None), r=turn(positions=None), out=None) == OK
    assert call(tokens=0, r=None, ax=None, x=heads(None), out=None) == OK


def test_norm_write_refused(L):  # noqa: F811
    def call(c=cache(), k=heads(), v=heads(), dtype=BF16, tokens=3, slots=FAKE, qw=norm(), kw=norm(), r=turn(), ax=axes(),
             q=heads(), qn=8, out=FAKE * 2, ot=1024, oh=128):
        return L.exl3_norm_kv_write(c, k, v, dtype, tokens, slots, qw, kw, r, ax, q, qn, out, ot, oh, None)

    for c in BAD_CACHES:
        assert call(c=c) == EINVAL
    for h in BAD_HEADS:
        assert call(k=h) == call(v=h) == call(q=h) == EINVAL
    for r in BAD_TURNS:
        assert call(r=r) == EINVAL
    for w in BAD_NORMS:
        assert call(qw=w) == call(kw=w) == EINVAL
    for ax in BAD_AXES:
        assert call(ax=ax) == EINVAL
    assert call(r=None) == EINVAL                             # axes of no rotation
    assert call(r=None, ax=None, qw=None) == EINVAL           # q with nothing to do
    assert call(qn=0, q=None, out=None) == EINVAL             # a norm of no q
    assert call(slots=None) == call(out=None) == call(tokens=-1) == call(dtype=5) == call(out=FAKE, oh=256) == EINVAL
    assert call(c=cache(fmt=0)) == call(c=cache(fmt=1), dtype=F16) == EINVAL
    assert call(c=cache(dim=192)) == EUNSUPPORTED
    assert call(tokens=0, k=heads(None), v=heads(None), slots=None, q=heads(None), out=None) == OK


def test_shared_refused(L):  # noqa: F811
    always = E.SHARE_ALWAYS

    def call(q=heads(), dtype=BF16, total=4, h=8, c=cache(), table=FAKE, width=40, cu=FAKE, lens=FAKE, batch=4, groups_at=FAKE,
             prefix=FAKE, groups=1, max_q=1, max_kv=64, max_prefix=always, scale=1.0, out=FAKE * 2, ot=1024, oh=128,
             ws=FAKE * 4, ws_bytes=1 << 40):
        return L.exl3_attention_shared(q, dtype, total, h, c, table, width, cu, lens, batch, groups_at, prefix, groups, max_q,
                                       max_kv, max_prefix, scale, out, ot, oh, ws, ws_bytes, None)

    for h in BAD_HEADS:
        assert call(q=h) == EINVAL
    for c in BAD_CACHES:
        assert call(c=c) == EINVAL
    for name in ("table", "cu", "lens", "groups_at", "prefix"):
        for p in MISALIGNED:
            assert call(**{name: p}) == EINVAL, name
    assert call(total=-1) == call(batch=-1) == call(groups=-1) == call(max_prefix=-1) == call(dtype=3) == call(h=5) == EINVAL
    assert call(width=0) == call(width=1 << 27) == call(max_q=0) == call(max_kv=-1) == EINVAL
    for s in (0.0, -2.0, math.nan, math.inf):
        assert call(scale=s) == EINVAL
    assert call(out=None) == call(out=FAKE, ot=2048) == call(ot=3) == EINVAL
    assert call(c=cache(fmt=0)) == call(c=cache(fmt=1), dtype=F16) == EINVAL
    assert call(c=cache(dim=32)) == EUNSUPPORTED
    for mp in (always, 300):  # shared, and the paged call that it else is
        need = L.exl3_attention_shared_workspace_bytes(4, 4, 1, 8, 2, 128, BF16, 3, 1, 64, mp)
        assert need > 0
        assert call(max_prefix=mp, ws=None) == call(max_prefix=mp, ws=FAKE + 8) == EINVAL
        assert call(max_prefix=mp, ws_bytes=need - 1) == EWORKSPACE
    assert call(total=0, q=heads(None), out=None, table=None, cu=None, lens=None, groups_at=None, prefix=None, ws=None,
                ws_bytes=0) == OK
    assert call(batch=0) == OK
    assert call(total=1 << 22, h=64, q=heads(token=64 * 128), ot=64 * 128) == EUNSUPPORTED  # more CTAs than a grid has


def test_shared_workspace_bytes(L):  # noqa: F811
    def size(total=64, batch=64, groups=1, h=32, kv=8, d=128, dtype=BF16, fmt=1, max_q=1, max_kv=9000, max_prefix=8192):
        return L.exl3_attention_shared_workspace_bytes(total, batch, groups, h, kv, d, dtype, fmt, max_q, max_kv, max_prefix)

    assert size(total=0) == size(batch=0) == size(h=7) == size(d=96) == size(max_q=0) == size(max_prefix=-1) == 0
    paged = L.exl3_attention_paged_workspace_bytes(64, 64, 32, 8, 128, 1, 9000, 0)
    assert size(groups=0) == size(max_prefix=100) == size(groups=64) == paged
    few = L.exl3_attention_paged_workspace_bytes(2, 2, 32, 8, 128, 1, 9000, 0)
    assert size(total=2, batch=2) == few            # two sequences behind 8192 keys do not pay
    assert size() > 0 and size() != paged           # 64 do
    assert size(fmt=2) == size(fmt=3) == size()
    assert size(dtype=F16, fmt=2) == paged          # but not in one fp16 term where the paged call has two
    assert size(total=2, batch=2, max_prefix=E.SHARE_ALWAYS) > few
    # bounded whatever the lengths: one wave of items, single tokens' own results and two of each CTA
    for kv_len in (1000, 1 << 20, 1 << 30):
        assert size(max_kv=kv_len, max_prefix=E.SHARE_ALWAYS) < 64 << 20


# ---------------------------------------------------------------- the binding's own checks


@pytest.fixture
def on_cpu(monkeypatch):
    """Checks of arguments without the demand for a GPU; the library's calls are recorded instead."""
    reached = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: reached.append(name) or 0

    monkeypatch.setattr(B, "_need", lambda t, dtype, name: None)
    monkeypatch.setattr(B, "_heads", lambda t, dtype, name: B._Heads(FAKE, 128, 64))
    monkeypatch.setattr(B, "_out_like", lambda x, out, name: (x, B._Heads(FAKE, 128, 64)))
    monkeypatch.setattr(B, "_raw_stream", lambda index: None)
    monkeypatch.setattr(B, "_shared_workspace_bytes", lambda *sizes: 16)
    monkeypatch.setattr(B, "lib", lambda: Library())
    return reached


def ints(*shape, dtype=torch.int32, device="cpu"):
    return torch.zeros(shape, dtype=dtype, device=device)


def rows(n=2, h=2, d=64, device="cpu"):
    return torch.zeros((n, h, d), dtype=torch.bfloat16, device=device)


def some_tables(device="cpu"):
    return B.KVTables(ints(3, 4, device=device), ints(3, device=device), ints(3, device=device), ints(9, device=device),
                      ints(1, device=device), 16)


def test_tables_refuse(on_cpu):
    t = some_tables()
    with pytest.raises(AttributeError):
        t.kv_lens = t.held
    lens = ints(6)
    good = dict(block_table=ints(3, 4), kv_lens=ints(3), held=ints(3), free_pages=ints(9), free_count=ints(1), page_size=16)
    for bad in (dict(block_table=ints(3)), dict(block_table=ints(3, 0)), dict(kv_lens=ints(2)), dict(held=ints(4)),
                dict(free_pages=ints(0)), dict(free_count=ints(2)), dict(page_size=24), dict(kv_lens=lens[:3], held=lens[1:4]),
                dict(held=ints(3, device="meta"))):
        with pytest.raises(ValueError):
            B.KVTables(**{**good, **bad})
    made = B.KVTables.empty(5, 100, 7, 16, device="cpu")
    assert made.block_table.shape == (5, 7) and made.free_pages.tolist() == [6, 5, 4, 3, 2, 1, 0]
    assert int(made.free_count) == 7 and not made.kv_lens.any() and not made.held.any()


def test_plan_checks(on_cpu):
    t = some_tables()
    cu, positions, slots, granted = E.kv_plan(t, ints(3), 7)
    assert on_cpu == ["exl3_kv_plan"]
    assert (cu.shape, positions.shape, slots.shape, granted.shape) == ((4,), (7,), (7,), (3,))
    assert (cu.dtype, positions.dtype, slots.dtype, granted.dtype) == (torch.int32, torch.int32, torch.int64, torch.bool)
    into = B.KVTables(t.block_table, ints(3), ints(3), t.free_pages, ints(1), 16)
    E.kv_plan(t, ints(3), 7, into=into)
    E.kv_plan(t, ints(3), 7, into=B.KVTables(t.block_table, t.kv_lens, ints(3), t.free_pages, t.free_count, 16))
    E.kv_release(t, ints(3, dtype=torch.bool), into=into)
    on_cpu.clear()
    wide = ints(20)
    shifted = B.KVTables(t.block_table, t.held, ints(3), t.free_pages, ints(1), 16)  # lengths where the pages held lie
    bad = [lambda: E.kv_plan(t, ints(2), 7), lambda: E.kv_plan(t, ints(3), 7, into=some_tables()),
           lambda: E.kv_plan(t, ints(3), 7, into=shifted), lambda: E.kv_plan(t, ints(3), 7, cu_q=ints(3)),
           lambda: E.kv_plan(t, ints(3), 7, positions=ints(8)), lambda: E.kv_plan(t, ints(3), 7, slots=ints(6, dtype=torch.int64)),
           lambda: E.kv_plan(t, ints(3), 7, granted=ints(2, dtype=torch.bool)),
           lambda: E.kv_plan(t, ints(3), 7, cu_q=wide[:4], positions=wide[3:10]),
           lambda: E.kv_plan(t, ints(3), 3, positions=t.kv_lens), lambda: E.kv_plan(t, wide[:3], 7, positions=wide[:7]),
           lambda: E.kv_plan(t, ints(3, device="meta"), 7), lambda: E.kv_plan(t, ints(3), 7, cu_q=ints(4, device="meta")),
           lambda: E.kv_release(t, ints(2, dtype=torch.bool)), lambda: E.kv_release(t, ints(3, dtype=torch.bool), shared=ints(4)),
           lambda: E.kv_release(t, ints(3, dtype=torch.bool), into=shifted),
           lambda: E.kv_release(t, ints(3, dtype=torch.bool, device="meta"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert not on_cpu


def test_norm_checks(on_cpu):
    phases, positions = ints(16, dtype=torch.int64), ints(2)
    two, which = ints(2, 2), ints(16, dtype=torch.uint8)
    w = torch.zeros(64, dtype=torch.bfloat16)
    E.rope(rows(), positions, phases)
    E.rope(rows(), two, phases, axes=which)
    E.rope(rows(), positions, phases, weight=w)
    E.rope(rows(), two, phases, axes=which, weight=w.expand(2, 64))
    c = B.KVCache.empty(3, 16, 2, 64, "int8", device="cpu")
    slots = ints(2, dtype=torch.int64)
    E.kv_write(c, rows(), rows(), slots)
    E.kv_write(c, rows(), rows(), slots, k_weight=w)
    E.kv_write(c, rows(), rows(), slots, q=rows(), q_weight=w)
    E.kv_write(c, rows(), rows(), slots, q=rows(), positions=two, phases=phases, axes=which)
    assert on_cpu == ["exl3_rope"] + ["exl3_norm_rope"] * 3 + ["exl3_kv_write"] + ["exl3_norm_kv_write"] * 3
    on_cpu.clear()
    bad = [lambda: E.rope(rows(), two, phases), lambda: E.rope(rows(), positions, phases, axes=which),
           lambda: E.rope(rows(), ints(2, 3), phases, axes=which), lambda: E.rope(rows(), two, phases, axes=which[:9]),
           lambda: E.rope(rows(), ints(0, 2), phases, axes=which), lambda: E.rope(rows(), positions, phases, weight=w[:32]),
           lambda: E.rope(rows(), positions, phases, weight=w.expand(3, 64)),
           lambda: E.rope(rows(), positions, phases, weight=w.to("meta")),
           lambda: E.rope(rows(), two, phases, axes=which.to("meta")),
           lambda: E.kv_write(c, rows(), rows(), slots, axes=which), lambda: E.kv_write(c, rows(), rows(), slots, q_weight=w),
           lambda: E.kv_write(c, rows(), rows(), slots, q=rows()), lambda: E.kv_write(c, rows(), rows(), slots, k_weight=w[:8]),
           lambda: E.kv_write(c, rows(), rows(), slots, k_weight=w.to("meta"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert not on_cpu


def test_shared_checks(on_cpu):
    c = B.KVCache.empty(3, 16, 2, 64, "int8", device="cpu")
    good = dict(q=rows(), cache=c, block_table=ints(2, 3), cu_q=ints(3), kv_lens=ints(2), cu_groups=ints(2), prefix_lens=ints(1),
                max_q=1, max_kv=9, max_prefix=9)
    E.attention_shared(**good)
    assert on_cpu == ["exl3_attention_shared"]
    on_cpu.clear()
    for bad in (dict(q=rows(d=128)), dict(cu_q=ints(0)), dict(kv_lens=ints(3)), dict(block_table=ints(3, 3)), dict(block_table=ints(2)),
                dict(cu_groups=ints(0)), dict(cu_groups=ints(3)), dict(prefix_lens=ints(2)), dict(cu_groups=ints(1, 2)),
                dict(cu_groups=ints(2, device="meta")), dict(prefix_lens=ints(1, device="meta")),
                dict(workspace=ints(16, dtype=torch.uint8, device="meta"))):
        with pytest.raises(ValueError):
            E.attention_shared(**{**good, **bad})
    assert not on_cpu


# ---------------------------------------------------------------- the oracle's norm


def test_oracle_norm_closed_forms():
    x = np.random.default_rng(1).standard_normal((4, 3, 16))
    w = np.random.default_rng(2).standard_normal(16)
    y, same = A.norm_rope(x, w, 0.0, None, None, None, "half", 1.0)
    assert y is same
    np.testing.assert_allclose((((y / w) ** 2).mean(-1)), 1.0)
    np.testing.assert_allclose(y, A.norm_rope(1e5 * x, w, 0.0, None, None, None, "half", 1.0)[0])
    np.testing.assert_allclose(A.norm_rope(1e-9 * x, w, 1.0, None, None, None, "half", 1.0)[0], 1e-9 * x * w)
    # one axis is the rotation of the normed row; an axis of zeros leaves its pairs alone
    words = [int(t * 2**64) for t in (0.16, 0.05, 0.02, 0.01, 0.005, 0.001, 0.0003, 0.0001)]
    p = np.array([[3, 5, 7, 9], [0, 0, 0, 0]])
    for layout in ("half", "interleaved"):
        z, row = A.norm_rope(x, w, 1e-6, p, [0] * 8, words, layout, 1.25)
        np.testing.assert_allclose(z, A.rope(row, p[0], words, layout, 1.25))
        z, row = A.norm_rope(x, w, 1e-6, p, [0, 1] * 4, words, layout, 1.0)
        second = np.arange(1, 8, 2)
        places = np.concatenate([second, second + 8]) if layout == "half" else np.concatenate([2 * second, 2 * second + 1])
        np.testing.assert_allclose(z[..., places], row[..., places])
        np.testing.assert_allclose((z**2).sum(-1), (row**2).sum(-1))  # turns keep the length
