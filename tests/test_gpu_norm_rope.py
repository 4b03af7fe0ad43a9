"""Norms of heads and rotary positions of several axes against the FP64 oracle, alone and with the cache write."""
import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0**-8, "f16": 2.0**-11}


def f64(t):
    return t.double().cpu().numpy()


def words(phases):
    return [int(p) % 2**64 for p in phases.cpu().tolist()]


def inputs(tokens, rows, dim, dtype, seed, pad=8):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, rows * dim + pad), generator=g)
    x[:, 5] *= 30.0
    if tokens > 3:
        x[1] *= 1e-3
        x[2] = 0.0
        x[3] *= 100.0
    return x.to(DT[dtype]).to(DEV)


def weights(shape, dtype, seed):
    return (1 + 0.3 * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(DT[dtype]).to(DEV)


def pairs(n, layout):
    """Index arrays of the first and second values of the rotated pairs."""
    return (np.arange(n), np.arange(n) + n) if layout == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)


def assert_normed(got, x, weight, eps, positions, axes, phases, layout, amplitude, dtype):
    """The norm: D squares summed in fp32 in any order, D 2^-24 at the most of a sum of positive terms, half of it after the
    root; its mean, the added eps, the root (2 ulp) and two products: 2^-21.  Then as a rotation of that row: 2^-20 of
    |a| + |b|; and one rounding to the type."""
    want, size = A.norm_rope(x, weight, eps, positions, axes, None if phases is None else words(phases), layout, amplitude)
    d = x.shape[-1]
    rel = d * 2.0**-25 + 2.0**-21
    mag = np.abs(size)
    tol = mag * rel
    if phases is not None:
        first, second = pairs(phases.numel(), layout)
        both = amplitude * (mag[..., first] + mag[..., second]) * (rel + 2.0**-20)
        tol[..., first] = tol[..., second] = both
    tol = tol * (1 + U[dtype]) + U[dtype] * np.abs(want) + (2.0**-25 if dtype == "f16" else 1e-38)
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def places(tokens, n_axes, rot, seed, kind):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 1 << 20, (n_axes, tokens), generator=g, dtype=torch.int32)
    p[0, 0] = 2**31 - 1
    if tokens > 1:
        p[-1, 1] = -3
    if kind == "sections":
        axes = (torch.arange(rot // 2) * n_axes // (rot // 2)).to(torch.uint8)
    else:
        axes = (torch.arange(rot // 2) % n_axes).to(torch.uint8)
    return p, axes


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,rot,n_axes", [(1, 1, 64, 16, 1), (7, 5, 128, 128, 3), (130, 3, 64, 64, 2),
                                                         (33, 41, 128, 48, 3), (700, 6, 128, 96, 2), (5, 2, 128, 16, 4)])
@pytest.mark.parametrize("each", [False, True])
def test_norm_rope(layout, dtype, tokens, heads, dim, rot, n_axes, each):
    x = inputs(tokens, heads + 1, dim, dtype, 11)
    view = x[:, :heads * dim].view(tokens, heads, dim)
    w = weights((heads, dim) if each else (dim,), dtype, 5)
    positions, axes = places(tokens, n_axes, rot, 3, "sections" if each else "turns")
    phases, amplitude = E.rope_phases(rot, scaling="yarn", factor=4.0)
    keep = x.clone()
    out = E.rope(view, positions.to(DEV), phases, layout, amplitude, axes=axes.to(DEV), weight=w, eps=1e-5)
    assert torch.equal(x, keep)
    args = (1e-5, positions.numpy(), axes.numpy(), phases, layout, amplitude, dtype)
    assert_normed(f64(out), f64(view), f64(w), *args)
    # in place, and into another strided place: the same bytes, nothing else touched
    other = torch.zeros_like(x)
    there = other[:, dim:(heads + 1) * dim].view(tokens, heads, dim)
    E.rope(view, positions.to(DEV), phases, layout, amplitude, out=there, axes=axes.to(DEV), weight=w, eps=1e-5)
    assert torch.equal(there, out) and not other[:, :dim].any() and not other[:, (heads + 1) * dim:].any()
    E.rope(view, positions.to(DEV), phases, layout, amplitude, out=view, axes=axes.to(DEV), weight=w, eps=1e-5)
    assert torch.equal(view, out) and torch.equal(x[:, heads * dim:], keep[:, heads * dim:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_axes_alone(layout):
    """Without a norm: the bytes of the rotation by each axis, pair by pair; a bad axis is taken as the last."""
    tokens, heads, dim, rot = 40, 3, 128, 96
    x = inputs(tokens, heads, dim, "bf16", 2, pad=0).view(tokens, heads, dim)
    positions, axes = places(tokens, 3, rot, 9, "turns")
    phases, amplitude = E.rope_phases(rot)
    axes[5] = 200
    got = E.rope(x, positions.to(DEV), phases, layout, amplitude, axes=axes.to(DEV))
    first, second = pairs(rot // 2, layout)
    rest = np.arange(rot, dim)
    assert torch.equal(got[..., rest], x[..., rest])
    for a in range(3):
        one = E.rope(x, positions[a].contiguous().to(DEV), phases, layout, amplitude)
        mine = np.minimum(axes.numpy(), 2) == a
        for side in (first, second):
            assert torch.equal(got[..., side[mine]], one[..., side[mine]])


@pytest.mark.parametrize("fmt", ["int8", "int4", "same"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,n_axes", [(1, 8, 2, 128, 128, 1), (9, 8, 8, 128, 48, 3), (300, 4, 2, 64, 64, 2),
                                                            (650, 3, 1, 128, 64, 3), (77, 0, 3, 64, 16, 2), (40, 6, 2, 64, 0, 1)])
@pytest.mark.parametrize("which", ["both", "q", "k"])
def test_norm_write(fmt, dtype, tokens, heads, kv, dim, rot, n_axes, which):
    """q's rows as the call alone makes them, keys as the 16-bit rows that this makes, quantised; values as they are."""
    if which == "q" and heads == 0:
        pytest.skip("no queries")
    if rot == 0 and which == "k":
        pytest.skip("queries that are neither normed nor rotated are not taken")
    fmt = dtype if fmt == "same" else fmt
    layout = "half" if tokens % 2 else "interleaved"
    x = inputs(tokens, heads + 2 * kv, dim, dtype, 5)
    q, k, v = (x[:, a * dim:b * dim].view(tokens, b - a, dim) for a, b in ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv)))
    qw = weights((dim,), dtype, 1) if which != "k" and heads else None
    kw = weights((kv, dim), dtype, 2) if which != "q" else None
    page = 16
    pages = tokens // page + 2
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:tokens].to(DEV)
    cache, plain = (E.KVCache.empty(pages, page, kv, dim, f) for f in (fmt, dtype))
    turn, args = {}, dict(eps=1e-6)
    if rot:
        positions, axes = places(tokens, n_axes, rot, 7, "sections")
        phases, amplitude = E.rope_phases(rot)
        turn = dict(positions=positions.to(DEV), phases=phases, layout=layout, amplitude=amplitude, axes=axes.to(DEV))
        oracle = (positions.numpy(), axes.numpy(), phases, layout, amplitude, dtype)
    else:
        oracle = (None, None, None, layout, 1.0, dtype)
    for c in (plain, cache):
        out = E.kv_write(c, k, v, slots, q=q if heads else None, q_weight=qw, k_weight=kw, **turn, **args)
        if heads:
            assert_normed(f64(out), f64(q), None if qw is None else f64(qw), 1e-6, *oracle)
        else:
            assert out is None
    rows, values = E.kv_read(plain, slots, dtype=DT[dtype])
    assert torch.equal(values, v)
    assert_normed(f64(rows), f64(k), None if kw is None else f64(kw), 1e-6, *oracle)
    if fmt != dtype:
        same = E.KVCache.empty(pages, page, kv, dim, fmt)
        E.kv_write(same, rows, v, slots)
        for a, b in ((cache.k, same.k), (cache.v, same.v), (cache.k_scale, same.k_scale), (cache.v_scale, same.v_scale)):
            assert torch.equal(a, b)


def test_rows_that_are_not_finite_stay_their_own():
    tokens, dim = 6, 128
    x = inputs(tokens, 2, dim, "bf16", 1, pad=0).view(tokens, 2, dim)
    x[1, 0, 3], x[2, 1, 9] = float("nan"), float("inf")
    positions = torch.arange(tokens, dtype=torch.int32, device=DEV)
    phases, amplitude = E.rope_phases(dim)
    w = weights((dim,), "bf16", 3)
    got = E.rope(x, positions, phases, weight=w)
    assert torch.isnan(got[1, 0]).all()
    clean = x.clone()
    clean[1, 0], clean[2, 1] = 0.0, 0.0
    want = E.rope(clean, positions, phases, weight=w)
    other = torch.ones((tokens, 2), dtype=torch.bool, device=DEV)
    other[1, 0] = other[2, 1] = False
    assert torch.equal(got[other], want[other])
    assert not want[1, 0].any()


def test_no_tokens():
    phases, _ = E.rope_phases(64)
    x = torch.empty((0, 3, 64), dtype=torch.bfloat16, device=DEV)
    out = E.rope(x, torch.empty((2, 0), dtype=torch.int32, device=DEV), phases,
                 axes=torch.zeros(32, dtype=torch.uint8, device=DEV), weight=weights((64,), "bf16", 1))
    assert out.shape == x.shape
