"""Rotary positions and the paged cache's rows against the FP64 oracle."""
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


def fused(tokens, heads, dim, dtype, seed, pad=8):
    """A fused projection's rows, wider than the heads asked for."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn((tokens, heads * dim + pad), generator=g).to(DT[dtype]).to(DEV)


def assert_rotated(got, x, positions, phases, layout, amplitude, dtype):
    """fp32 steps: the angle is off by 2^-25 pi at the most by its rounding and 2^-31 pi by the phase's cut, cosine and
    sine by 2 ulp, each product and the sum by one rounding: 2^-20 of |a| + |b|; then one rounding to the type."""
    want = A.rope(x, positions, words(phases), layout, amplitude)
    n = 2 * phases.numel()
    mag = np.abs(x)
    half = mag[..., :n // 2] + mag[..., n // 2:n] if layout == "half" else mag[..., 0:n:2] + mag[..., 1:n:2]
    pair = np.zeros_like(mag)
    if layout == "half":
        pair[..., :n // 2] = pair[..., n // 2:n] = half
    else:
        pair[..., 0:n:2] = pair[..., 1:n:2] = half
    tol = amplitude * pair * 2.0**-20
    tol = tol * (1 + U[dtype]) + U[dtype] * np.abs(want) + 2.0**-25
    tol[..., n:] = 0
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 64, 16), (7, 5, 128, 128), (130, 3, 64, 64), (33, 41, 128, 48),
                                                  (700, 6, 128, 96), (5, 2, 128, 16)])
def test_rope(layout, dtype, tokens, heads, dim, rot):
    x = fused(tokens, heads + 1, dim, dtype, 11)
    view = x[:, :heads * dim].view(tokens, heads, dim)
    g = torch.Generator().manual_seed(3)
    positions = torch.randint(0, 1 << 20, (tokens,), generator=g, dtype=torch.int32)
    positions[0] = 2**31 - 1
    if tokens > 2:
        positions[1], positions[2] = 0, 1
    phases, amplitude = E.rope_phases(rot, scaling="yarn", factor=4.0)
    keep = x.clone()
    out = E.rope(view, positions.to(DEV), phases, layout, amplitude)
    torch.cuda.synchronize()
    assert torch.equal(x, keep)
    assert_rotated(f64(out), f64(view), positions.tolist(), phases, layout, amplitude, dtype)
    # in place, and into another strided place: the same bytes, nothing else touched
    other = torch.zeros_like(x)
    E.rope(view, positions.to(DEV), phases, layout, amplitude, out=other[:, dim:(heads + 1) * dim].view(tokens, heads, dim))
    E.rope(view, positions.to(DEV), phases, layout, amplitude, out=view)
    assert torch.equal(view, out)
    assert torch.equal(other[:, dim:(heads + 1) * dim].reshape(tokens, heads, dim), out)
    assert torch.equal(x[:, heads * dim:], keep[:, heads * dim:])
    assert not other[:, :dim].any() and not other[:, (heads + 1) * dim:].any()


@pytest.mark.parametrize("fmt", ["int8", "int4", "same"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,kv,dim,page", [(1, 1, 64, 16), (9, 8, 128, 16), (300, 2, 128, 64), (77, 3, 64, 256),
                                                (650, 1, 128, 32)])
def test_write_and_read(fmt, dtype, tokens, kv, dim, page):
    """The bytes that land in the cache are the oracle's, and nothing else in it changes."""
    fmt = dtype if fmt == "same" else fmt
    x = fused(tokens, 2 * kv, dim, dtype, 5)
    x[:, 3] *= 40.0  # a channel that stands out
    if tokens > 4:
        x[2, :2 * kv * dim] = 0.0       # rows of zeros
        x[3, 0], x[3, kv * dim] = float("inf"), float("nan")  # rows that are not finite
        x[4, :2 * kv * dim] = 1e-7 if dtype == "f16" else 1e-38
    k, v = x[:, :kv * dim].view(tokens, kv, dim), x[:, kv * dim:2 * kv * dim].view(tokens, kv, dim)
    pages = tokens // page + 3
    cache = E.KVCache.empty(pages, page, kv, dim, fmt)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).random_(0, 256, generator=torch.Generator(device=DEV).manual_seed(1))
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:tokens]
    if tokens > 8:
        slots[5], slots[6], slots[7] = -1, pages * page, 2**40  # padding
    assert E.kv_write(cache, k, v, slots.to(DEV)) is None
    torch.cuda.synchronize()
    good = ((slots >= 0) & (slots < pages * page)).numpy()
    s = slots.numpy()
    want = [t.cpu().clone() for t in before]
    for side, rows in ((0, k), (1, v)):
        r = rows.cpu()
        if fmt in A.TOP:
            codes, scales = A.quantise(rows.float().cpu().numpy(), fmt)
            data = torch.tensor(A.stored(codes, fmt))
            bits = torch.tensor((scales.view(np.uint32) >> 16).astype(np.uint16).view(np.int16))
        for t in np.flatnonzero(good):
            p, o = int(s[t]) // page, int(s[t]) % page
            if fmt in A.TOP:
                want[side][p, :, o] = data[t]
                want[2 + side].view(torch.int16)[p, :, o] = bits[t]
            else:
                want[side][p, :, o] = r[t]
    now = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    for a, b in zip(now, want):
        a, b = a.cpu(), b
        nan = torch.isnan(a.float()) & torch.isnan(b.float()) if a.dtype == torch.bfloat16 and a.dim() == 3 else None
        same = a.view(torch.int16) == b.view(torch.int16) if a.dtype != torch.uint8 else a == b
        assert bool((same if nan is None else same | nan).all())
    # read back: one rounding of the value, exact before it up to the fp32 product's
    for out_dtype in ("bf16", "f16"):
        gk, gv = E.kv_read(cache, slots.to(DEV), dtype=DT[out_dtype])
        torch.cuda.synchronize()
        for got, rows in ((gk, k), (gv, v)):
            got = f64(got)
            assert not got[~good].any()
            if fmt in A.TOP:
                codes, scales = A.quantise(rows.float().cpu().numpy(), fmt)
                back = A.read_back(codes, scales)
            else:
                back = f64(rows)
            back, got = back[good], got[good]
            bad = ~np.isfinite(back)
            assert (np.isfinite(got) == ~bad)[np.abs(np.where(bad, 0, back)) < 6e4].all()
            fine = np.isfinite(back) & (np.abs(back) < 6e4)
            step = 2.0**-25 if out_dtype == "f16" else 1e-40
            assert (np.abs(got - back)[fine] <= (np.abs(back) * (U[out_dtype] + 2.0**-23) + step)[fine]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("fmt", ["int8", "int4", "bf16"])
@pytest.mark.parametrize("tokens", [1, 13, 200, 700])
def test_write_rotates_as_rope_does(layout, fmt, tokens):
    """The fused call's bytes are those of rope followed by a plain write; q in place too."""
    kv, heads, dim, page = 4, 12, 128, 32
    x = fused(tokens, heads + 2 * kv, dim, "bf16", 9, pad=0).view(tokens, heads + 2 * kv, dim)
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    phases, amplitude = E.rope_phases(64, scaling="ntk", factor=2.0)
    positions = torch.arange(1000, 1000 + tokens, dtype=torch.int32, device=DEV)
    slots = torch.randperm((tokens // page + 2) * page, generator=torch.Generator().manual_seed(1))[:tokens].to(DEV)
    one = E.KVCache.empty(tokens // page + 2, page, kv, dim, fmt)
    two = E.KVCache.empty(tokens // page + 2, page, kv, dim, fmt)
    qr = E.kv_write(one, k, v, slots, q=q, positions=positions, phases=phases, layout=layout, amplitude=amplitude)
    turned = E.rope(x[:, :heads + kv], positions, phases, layout, amplitude)
    E.kv_write(two, turned[:, heads:], v, slots)
    assert torch.equal(qr, turned[:, :heads])
    for a, b in ((one.k, two.k), (one.v, two.v), (one.k_scale, two.k_scale), (one.v_scale, two.v_scale)):
        assert a is None or torch.equal(a, b)
    E.kv_write(one, k, v, slots, q=q, positions=positions, phases=phases, layout=layout, amplitude=amplitude, q_out=q)
    assert torch.equal(q, qr)
    # keys alone
    E.kv_write(one, x[:, heads:heads + kv], v, slots, positions=positions, phases=phases, layout=layout, amplitude=amplitude)
    assert torch.equal(one.k, two.k)


def test_cache_beyond_32_bit_offsets():
    """Rows whose byte offset passes 2^32."""
    kv, dim, page = 8, 128, 256
    pages = 8400  # 4.4 GB a side
    cache = E.KVCache.empty(pages, page, kv, dim, "bf16")
    x = fused(40, 2 * kv, dim, "bf16", 4, pad=0).view(40, 2 * kv, dim)
    slots = torch.randint(0, pages * page, (40,), generator=torch.Generator().manual_seed(8))
    slots[0], slots[1] = pages * page - 1, 0
    assert slots.unique().numel() == 40
    E.kv_write(cache, x[:, :kv], x[:, kv:], slots.to(DEV))
    k, v = E.kv_read(cache, slots.to(DEV))
    assert torch.equal(k, x[:, :kv]) and torch.equal(v, x[:, kv:])
    page_, off = slots // page, slots % page
    assert torch.equal(cache.k[page_.to(DEV), :, off.to(DEV)], x[:, :kv])
    assert int((cache.v != 0).sum()) == int((x[:, kv:] != 0).sum())


def test_no_tokens_and_refusals():
    cache = E.KVCache.empty(2, 16, 2, 64, "int8")
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    E.kv_write(cache, none, none, ids)
    assert E.kv_read(cache, ids)[0].shape == (0, 2, 64)
    phases, amp = E.rope_phases(64)
    assert E.rope(none, torch.empty(0, dtype=torch.int32, device=DEV), phases).shape == (0, 2, 64)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    slots = torch.arange(4, device=DEV)
    with pytest.raises(ValueError):
        E.rope(x.float(), pos, phases)
    with pytest.raises(ValueError):
        E.rope(x, pos.long(), phases)
    with pytest.raises(ValueError):
        E.rope(x, pos[:3], phases)
    with pytest.raises(E.Exl3Error):
        E.rope(x, pos, E.rope_phases(72)[0])  # not a multiple of 16, more than the head
    with pytest.raises(E.Exl3Error):
        E.rope(torch.zeros((4, 2, 80), dtype=torch.bfloat16, device=DEV), pos, phases)  # head size
    with pytest.raises(E.Exl3Error):
        E.rope(torch.zeros((4, 132), dtype=torch.bfloat16, device=DEV)[:, :128].view(4, 2, 64), pos, phases)  # stride
    big = torch.zeros((8, 2, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        E.rope(big[:4], pos, phases, out=big[2:6])  # overlap
    with pytest.raises(ValueError):
        E.kv_write(cache, x, x, slots, q=x)  # q without positions
    with pytest.raises(ValueError):
        E.kv_write(cache, x, x, slots.int())
    with pytest.raises(ValueError):
        E.kv_write(cache, x[:, :1], x[:, :1], slots)
    with pytest.raises(E.Exl3Error):
        E.kv_write(E.KVCache.empty(2, 16, 2, 64, "f16"), x, x, slots)  # a 16-bit cache of another type
    with pytest.raises(E.Exl3Error):
        E.kv_write(E.KVCache.empty(2, 24, 2, 64, "int8"), x, x, slots)  # page size
    with pytest.raises(ValueError):
        E.KVCache(cache.k, cache.v, None, None, "int8")
    with pytest.raises(ValueError):
        E.kv_read(cache, slots, dtype=torch.float32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [16, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("dim,kv,heads,tokens", [(128, 1, 3, 5), (128, 3, 6, 170), (128, 24, 24, 3), (64, 5, 5, 650), (64, 8, 16, 9)])
def test_write_rotates_parts_of_heads(layout, rot, dim, kv, heads, tokens):
    """Every rotated width, with the partners of a pair near and far: the fused call against rope and a plain write."""
    if rot > dim:
        pytest.skip("no such width")
    x = fused(tokens, heads + 2 * kv, dim, "f16", 11, pad=0).view(tokens, heads + 2 * kv, dim)
    q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
    phases, amplitude = E.rope_phases(rot, scaling="linear", factor=3.0)
    positions = torch.arange(77, 77 + tokens, dtype=torch.int32, device=DEV)
    slots = torch.randperm((tokens // 16 + 2) * 16, generator=torch.Generator().manual_seed(3))[:tokens].to(DEV)
    turned = E.rope(x[:, :heads + kv], positions, phases, layout, amplitude)
    for fmt in ("f16", "int8", "int4"):
        one, two = (E.KVCache.empty(tokens // 16 + 2, 16, kv, dim, fmt) for _ in range(2))
        qr = E.kv_write(one, k, v, slots, q=q, positions=positions, phases=phases, layout=layout, amplitude=amplitude)
        E.kv_write(two, turned[:, heads:], v, slots)
        assert torch.equal(qr, turned[:, :heads])
        for a, b in ((one.k, two.k), (one.v, two.v), (one.k_scale, two.k_scale), (one.v_scale, two.v_scale)):
            assert a is None or torch.equal(a, b)
