"""Rotary, cache and attention calls without a GPU: phases against the oracle, workspace sizes, refusals on the host."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from exl3_trellis_quantized_gb300 import binding as B
from oracle import attention_oracle as A

FAKE = 1 << 20  # a 16-byte-aligned address; never dereferenced because validation fails first
OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, 1, 2, 3
F16, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    try:
        return B.lib()
    except ImportError as e:  # the build step must have run first
        pytest.fail(str(e))


# ---------------------------------------------------------------- phases


@pytest.mark.parametrize("rot", [2, 16, 64, 128])
@pytest.mark.parametrize("kind,args", [
    ("plain", {}), ("plain", {"base": 500000.0}), ("linear", {"factor": 4.0}), ("ntk", {"factor": 8.0}),
    ("yarn", {"factor": 16.0}), ("yarn", {"factor": 4.0, "fast": 16.0, "slow": 2.0, "original_len": 8192.0}),
])
def test_phases(rot, kind, args):
    if kind == "ntk" and rot == 2:
        with pytest.raises(E.Exl3Error):
            E.rope_phases(rot, scaling=kind, device="cpu", **args)
        return
    words, amplitude = E.rope_phases(rot, scaling=kind, device="cpu", **args)
    freq, amp = A.phases(rot, scaling=kind, **args)
    assert words.shape == (rot // 2,) and words.dtype == torch.int64
    turns = np.array([(int(w) % 2**64) / 2.0**64 for w in words])
    # 64-bit arithmetic on both sides, a power and a few products: some units of the last place; and one unit of 2^-64
    assert (np.abs(turns - freq / (2 * math.pi)) <= 2.0**-48 * turns + 2.0**-64).all()
    assert amplitude == pytest.approx(amp, rel=2.0**-23)
    assert turns[0] == pytest.approx(1 / (2 * math.pi) / (args["factor"] if kind == "linear" else 1), rel=1e-15)


def test_phases_refused(L):
    out, amp = torch.empty(64, dtype=torch.int64), ctypes.c_float()

    def call(rot=128, base=1e4, kind=0, factor=1.0, fast=32.0, slow=1.0, length=4096.0, dst=out.data_ptr()):
        return L.exl3_rope_phases(rot, base, kind, factor, fast, slow, length, dst, ctypes.byref(amp))

    assert call() == OK
    bad = [dict(rot=0), dict(rot=3), dict(rot=-2), dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(kind=4),
           dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=2, factor=math.inf), dict(kind=3, fast=1.0),
           dict(kind=3, slow=0.0), dict(kind=3, length=0.0), dict(dst=None)]
    for args in bad:
        assert call(**args) == EINVAL, args
    assert L.exl3_rope_phases(128, 1e4, 0, 1.0, 32.0, 1.0, 4096.0, out.data_ptr(), None) == EINVAL


# ---------------------------------------------------------------- refusals


def heads(data=FAKE, token=1024, head=128):
    return B._Heads(data, token, head)


def turn(phases=FAKE, positions=FAKE, rot=128, layout=0, amplitude=1.0):
    return B._Rope(phases, positions, rot, layout, amplitude)


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=10, page=16, kv=2, dim=128, fmt=3):
    return B._Cache(k, v, ks, vs, pages, page, kv, dim, fmt)


BAD_HEADS = [heads(None), heads(FAKE + 8), heads(token=1020), heads(head=4), heads(token=0), heads(head=-8),
             heads(token=1 << 32)]
BAD_TURNS = [turn(None), turn(FAKE + 4), turn(positions=None), turn(positions=FAKE + 2), turn(rot=8), turn(rot=24),
             turn(rot=144), turn(rot=0), turn(layout=2), turn(amplitude=math.nan), turn(amplitude=math.inf)]
BAD_CACHES = [cache(k=None), cache(v=FAKE + 8), cache(ks=None), cache(vs=FAKE + 2), cache(pages=0), cache(pages=1 << 31),
              cache(page=8), cache(page=24), cache(page=512), cache(kv=0), cache(kv=65537), cache(dim=0), cache(fmt=4),
              cache(fmt=-1), cache(pages=(1 << 30), kv=2)]


def test_rope_refused(L):
    def call(x=heads(), dtype=BF16, tokens=3, n=4, dim=128, r=turn(), out=FAKE * 2, ot=1024, oh=128):
        return L.exl3_rope(x, dtype, tokens, n, dim, r, out, ot, oh, None)

    for h in BAD_HEADS:
        assert call(x=h) == EINVAL
    for r in BAD_TURNS:
        assert call(r=r) == EINVAL
    assert call(x=None) == call(r=None) == call(out=None) == call(out=FAKE + 2) == EINVAL
    assert call(out=FAKE, ot=2048) == EINVAL  # in place with other strides
    assert call(tokens=-1) == call(tokens=1 << 40) == call(n=0) == call(n=65537) == call(dtype=2) == EINVAL
    assert call(ot=4) == call(oh=0) == call(dim=0) == EINVAL
    assert call(dim=96) == call(dim=256) == EUNSUPPORTED
    assert call(tokens=0, x=heads(None), r=turn(positions=None), out=None) == OK  # nothing to do


def test_kv_write_refused(L):
    def call(c=cache(), k=heads(), v=heads(), dtype=BF16, tokens=3, slots=FAKE, r=turn(), q=heads(), qn=8, out=FAKE * 2,
             ot=1024, oh=128):
        return L.exl3_kv_write(c, k, v, dtype, tokens, slots, r, q, qn, out, ot, oh, None)

    for c in BAD_CACHES:
        assert call(c=c) == EINVAL
    for h in BAD_HEADS:
        assert call(k=h) == call(v=h) == call(q=h) == EINVAL
    for r in BAD_TURNS:
        assert call(r=r) == EINVAL
    assert call(c=None) == call(k=None) == call(v=None) == call(q=None) == EINVAL
    assert call(r=None) == EINVAL  # q is only taken to be rotated
    assert call(slots=None) == call(slots=FAKE + 4) == call(out=None) == call(qn=-1) == call(qn=65537) == EINVAL
    assert call(tokens=-1) == call(dtype=5) == call(ot=7) == call(out=FAKE, oh=256) == EINVAL
    assert call(c=cache(fmt=0)) == call(c=cache(fmt=1), dtype=F16) == EINVAL  # a 16-bit cache of the other type
    assert call(c=cache(dim=192)) == EUNSUPPORTED
    assert call(tokens=0, k=heads(None), v=heads(None), slots=None, q=heads(None), out=None) == OK


def test_kv_read_refused(L):
    def call(c=cache(), slots=FAKE, tokens=3, dtype=BF16, k=FAKE, v=FAKE):
        return L.exl3_kv_read(c, slots, tokens, dtype, k, v, None)

    for c in BAD_CACHES:
        assert call(c=c) == EINVAL
    assert call(slots=None) == call(slots=FAKE + 4) == call(k=None) == call(v=FAKE + 8) == EINVAL
    assert call(tokens=-1) == call(dtype=2) == call(c=None) == EINVAL
    assert call(tokens=0, slots=None, k=None, v=None) == OK


def test_prompt_refused(L):
    def call(q=heads(), k=heads(), v=heads(), dtype=BF16, total=5, h=8, kv=2, dim=128, cu=FAKE, batch=1, window=0,
             scale=1.0, out=FAKE * 2, ot=1024, oh=128):
        return L.exl3_attention_prompt(q, k, v, dtype, total, h, kv, dim, cu, batch, window, scale, out, ot, oh, None)

    for h in BAD_HEADS:
        assert call(q=h) == call(k=h) == call(v=h) == EINVAL
    assert call(total=-1) == call(batch=-1) == call(dtype=2) == call(window=-1) == call(cu=None) == call(cu=FAKE + 2) == EINVAL
    assert call(h=7) == call(h=0) == call(kv=0) == call(h=258, kv=2) == EINVAL  # groups of whole heads, at most 128
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=s) == EINVAL
    assert call(out=None) == call(ot=0) == call(oh=12) == call(dim=0) == EINVAL
    assert call(dim=80) == EUNSUPPORTED
    assert call(total=0, q=heads(None), k=heads(None), v=heads(None), out=None, cu=None) == OK
    assert call(batch=0, cu=None) == OK


def test_paged_refused(L):
    big = 1 << 30

    def call(q=heads(), dtype=BF16, total=4, h=8, c=cache(), table=FAKE, width=4, cu=FAKE, lens=FAKE, batch=4, max_q=1,
             max_kv=64, window=0, scale=1.0, out=FAKE * 2, ot=1024, oh=128, ws=FAKE * 4, ws_bytes=big):
        return L.exl3_attention_paged(q, dtype, total, h, c, table, width, cu, lens, batch, max_q, max_kv, window, scale,
                                      out, ot, oh, ws, ws_bytes, None)

    for h in BAD_HEADS:
        assert call(q=h) == EINVAL
    for c in BAD_CACHES:
        assert call(c=c) == EINVAL
    assert call(total=-1) == call(batch=-1) == call(dtype=3) == call(h=5) == call(window=-3) == EINVAL
    for p in (None, FAKE + 2):
        assert call(table=p) == call(cu=p) == call(lens=p) == EINVAL
    assert call(width=0) == call(width=1 << 27) == call(max_q=0) == call(max_kv=-1) == EINVAL
    for s in (0.0, -2.0, math.nan, math.inf):
        assert call(scale=s) == EINVAL
    assert call(out=None) == call(out=FAKE, ot=2048) == call(ot=3) == EINVAL
    assert call(c=cache(fmt=0)) == call(c=cache(fmt=1), dtype=F16) == EINVAL
    assert call(c=cache(dim=32)) == EUNSUPPORTED
    need = L.exl3_attention_paged_workspace_bytes(4, 4, 8, 2, 128, 1, 64, 0)
    assert need > 0
    assert call(ws=None) == call(ws=FAKE + 8) == EINVAL
    assert call(ws_bytes=need - 1) == EWORKSPACE
    assert call(total=0, q=heads(None), out=None, table=None, cu=None, lens=None, ws=None, ws_bytes=0) == OK
    assert call(batch=0) == OK


# ---------------------------------------------------------------- workspace


def test_workspace_bytes():
    size = E.attention_paged_workspace_bytes
    assert size(0, 4, 8, 2, 128, 1, 64) == size(4, 0, 8, 2, 128, 1, 64) == 0
    # nothing that the call would refuse
    assert size(4, 4, 7, 2, 128, 1, 64) == size(4, 4, 8, 2, 96, 1, 64) == size(4, 4, 8, 2, 128, 0, 64) == 0
    # single tokens: two partial results of 16 rows for every CTA, whatever the lengths
    one = size(1, 1, 8, 2, 128, 1, 1)
    assert one % (2 * 16 * (128 + 2) * 4) == 0
    last = 0
    for kv in (1, 100, 1000, 10000, 100000, 1 << 20):
        now = size(8, 8, 32, 8, 128, 1, kv)
        assert last <= now <= 152 * 8 * 2 * 16 * (128 + 2) * 4
        last = now
    # many rows fill the GPU by themselves: no parts; few over long keys: parts of every row's fp32 result
    assert size(8192, 1, 32, 8, 128, 8192, 8192) == 0
    few = size(100, 1, 8, 1, 128, 100, 100000)
    assert few > 0 and few % (100 * 8 * (128 + 2) * 4) == 0 and few // (100 * 8 * (128 + 2) * 4) <= 16
    # a window bounds the keys that are worth parting
    assert size(100, 1, 8, 1, 128, 100, 100000, 64) == 0


# ---------------------------------------------------------------- binding's own checks (no library call reached)


def test_binding_refuses():
    x = torch.zeros(2, 3, 128, dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)):
        E.rope(x.float(), torch.zeros(2, dtype=torch.int32), torch.zeros(64, dtype=torch.int64))
    with pytest.raises(KeyError):
        E.rope_phases(128, scaling="other", device="cpu")
    with pytest.raises(ValueError):
        E.KVCache.empty(4, 16, 2, 128, "int3", device="cpu")


# ---------------------------------------------------------------- the oracle itself


def test_oracle_rotation_closed_forms():
    x = np.random.default_rng(1).standard_normal((3, 2, 16))
    quarter = [2**62] * 8  # a quarter of a turn a position
    for layout in ("half", "interleaved"):
        y = A.rope(x, [0, 1, 2], quarter, layout, 1.0)
        a, b = ((x[..., :8], x[..., 8:]) if layout == "half" else (x[..., 0::2], x[..., 1::2]))
        c, d = ((y[..., :8], y[..., 8:]) if layout == "half" else (y[..., 0::2], y[..., 1::2]))
        np.testing.assert_allclose(c[0], a[0], atol=1e-15)
        np.testing.assert_allclose(c[1], -b[1], atol=1e-15)
        np.testing.assert_allclose(d[1], a[1], atol=1e-15)
        np.testing.assert_allclose(c[2], -a[2], atol=1e-15)
    # scores depend on the distance of positions only
    words = [int(t * 2**64) for t in (0.1591, 0.01, 0.003, 0.0001, 0.2, 0.05, 0.007, 0.0009)]
    q, k = x[:1], x[1:2]
    score = [float((A.rope(q, [p], words, "half", 1.0) * A.rope(k, [p - 5], words, "half", 1.0)).sum()) for p in (5, 77, 4000)]
    np.testing.assert_allclose(score, score[0], rtol=1e-10)


@pytest.mark.parametrize("fmt", ["int8", "int4"])
def test_oracle_quantiser(fmt):
    x = np.random.default_rng(2).standard_normal((50, 128)).astype(np.float32)
    codes, scales = A.quantise(x, fmt)
    assert np.abs(codes).max() <= A.TOP[fmt] and (np.abs(codes).max(-1) >= A.TOP[fmt] - 1).all()
    assert (A.codes_of(A.stored(codes, fmt), fmt) == codes).all()
    # half a step an entry in the rotated basis is, transformed back, at most half a step of all D entries
    err = np.abs(A.read_back(codes, scales) - x).max(-1)
    assert (err <= 0.51 * scales * 8).all()
    zero, one = A.quantise(np.zeros((1, 64), np.float32), fmt)
    assert not zero.any() and one[0] == 1.0
    bad, nan = A.quantise(np.array([[np.inf] + [0.0] * 63], np.float32), fmt)
    assert not bad.any() and np.isnan(nan[0])


def test_oracle_attention_closed_forms():
    v = np.random.default_rng(3).standard_normal((6, 1, 64))
    zero = np.zeros((6, 2, 64))
    out, spread, _ = A.attention(zero, zero[:, :1], v)
    for t in range(6):  # equal scores: the mean of what is seen
        np.testing.assert_allclose(out[t, 1], v[:t + 1, 0].mean(0))
        np.testing.assert_allclose(spread[t, 0], np.abs(v[:t + 1, 0]).mean(0))
    out, _, _ = A.attention(zero, zero[:, :1], v, window=1)
    np.testing.assert_allclose(out[:, 0], v[:, 0])
    out, _, _ = A.attention(zero[:2], zero[:, :1], v)  # the last two of six tokens
    np.testing.assert_allclose(out[0, 0], v[:5, 0].mean(0))
    out, _, _ = A.attention(zero[:2], zero[:1, :1], v[:1])  # more query tokens than keys: the first sees nothing
    assert not out[0].any()
    np.testing.assert_allclose(out[1, 0], v[0, 0])


def test_paged_refuses_more_items_than_a_grid(L):
    """Sequences times key heads index one axis of a grid, also where most sequences are empty."""
    kv, batch = 1024, 1 << 22
    need = L.exl3_attention_paged_workspace_bytes(4, batch, kv, kv, 128, 1, 64, 0)
    st = L.exl3_attention_paged(heads(token=kv * 128), BF16, 4, kv, cache(kv=kv), FAKE, 4, FAKE, FAKE, batch, 1, 64, 0, 1.0,
                                FAKE * 2, kv * 128, 128, FAKE * 4, need, None)
    assert st == EUNSUPPORTED
