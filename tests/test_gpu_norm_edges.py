"""Norms of heads without a rotation (against the FP64 oracle), and rows without a norm beside rows with one."""
import pytest
import torch

import exl3_trellis_quantized_gb300 as E
from test_gpu_norm_rope import DEV, DT, assert_normed, f64, inputs, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 64), (7, 5, 128), (130, 3, 64), (33, 41, 128), (700, 6, 128)])
@pytest.mark.parametrize("each", [False, True])
def test_norm_without_a_rotation(layout, dtype, tokens, heads, dim, each):
    x = inputs(tokens, heads + 1, dim, dtype, 11)
    view = x[:, :heads * dim].view(tokens, heads, dim)
    w = weights((heads, dim) if each else (dim,), dtype, 5)
    keep = x.clone()
    out = E.rope(view, layout=layout, weight=w, eps=1e-5)
    assert torch.equal(x, keep)
    assert_normed(f64(out), f64(view), f64(w), 1e-5, None, None, None, layout, 1.0, dtype)
    E.rope(view, layout=layout, out=view, weight=w, eps=1e-5)
    assert torch.equal(view, out) and torch.equal(x[:, heads * dim:], keep[:, heads * dim:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,rot", [(128, 48), (64, 16), (128, 128), (64, 64)])
@pytest.mark.parametrize("normed", ["q", "k"])
def test_what_does_not_turn_stays(layout, dtype, dim, rot, normed):
    """Rows without a norm beside rows with one: values that do not turn come out as they are, whatever stands beside them,
    and pairs that turn take no more than each other."""
    tokens, heads, kv = 9, 3, 2
    x = inputs(tokens, heads + 2 * kv, dim, dtype, 5, pad=0).view(tokens, heads + 2 * kv, dim)
    q, k, v = x.split([heads, kv, kv], dim=1)
    plain = q if normed == "k" else k
    clean = plain.clone()
    bad = [(1, 0, dim - 1, float("inf")), (2, 1, dim - 6, float("nan")), (4, 0, rot - 1, float("-inf"))]
    for t, h, d, value in bad:
        plain[t, h, d] = value
    w = weights((dim,), dtype, 1)
    page, pages = 16, 3
    slots = torch.arange(tokens, device=DEV) + 5
    phases, amplitude = E.rope_phases(rot)
    positions = torch.arange(tokens, dtype=torch.int32, device=DEV) * 7

    def write(rows):
        cache = E.KVCache.empty(pages, page, kv, dim, dtype)
        turn = dict(positions=positions, phases=phases, layout=layout, amplitude=amplitude)
        if normed == "k":
            return E.kv_write(cache, k, v, slots, q=rows, k_weight=w, **turn)
        E.kv_write(cache, rows, v, slots, q=q, q_weight=w, **turn)
        return E.kv_read(cache, slots, dtype=DT[dtype])[0]

    got, want = write(plain), write(clean)
    both = torch.zeros_like(got, dtype=torch.bool)
    for t, h, d, value in bad:
        pair = [d]
        if d < rot:
            pair.append((d + rot // 2) % rot if layout == "half" else d ^ 1)
        both[t, h, pair] = True
        if d >= rot:
            assert torch.equal(got[t, h, d].isnan(), plain[t, h, d].isnan())
            assert value != value or float(got[t, h, d]) == value
        else:
            assert not torch.isfinite(got[t, h, pair]).any()
    assert torch.equal(got[~both], want[~both])
    assert torch.equal(want[..., rot:], clean[..., rot:])
