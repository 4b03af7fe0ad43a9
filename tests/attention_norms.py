"""How far a row of attention's output may be off in norm: a bound close enough to the real error that a lost key tile shows.

attention_check bounds every entry by the worst case, which over a quantised cache (rotated rows, D entries' errors summed)
is larger than many outputs.  Rounding errors of different keys are independent, so the error of a row is near the root of
the sum of their squares; this takes four times that root, with every rounding at its largest (u where the mean square is
u^2 / 3: seven standard deviations), and adds what is not independent:

  weight j (w_j of the definition, sum 1) rounds by u_p w_j, times the norm of v_j;
  its score is off by e_j, which moves the row by w_j e_j |v_j - o|: over a quantised cache by the fp16 roundings of q and
    of the keys in the rotated basis, entry by entry, e_j^2 = scale^2 2 u^2 sum_d (q_d k_jd)^2; by fp32 sums and the
    exponent's own roundings, 2^-20 (1 + scale sum_d |q_d k_jd|);
  values over a quantised cache round by u_v |v_j|;
  weights below fp16's normal range are off by 2^-25 of the largest weight's;
  the sum of the weights is fp32 (2^-20), and the result rounds to its type.
"""
import numpy as np

from attention_check import U
from oracle import attention_oracle as A


def bound(q, k, v, window, scale, dtype, fmt):
    """(out [Lq, H, D], tolerance [Lq, H] of a row's norm) of one sequence, 64 bits; k, v as read back for int8/int4."""
    lq, h, d = q.shape
    lk, kv, _ = k.shape
    scale = d**-0.5 if scale is None else scale
    quant = fmt in A.TOP
    u = 2.0**-11 if quant else 0.0
    out, _, _ = A.attention(q, k, v, window, scale)
    if quant:
        hm = A.hadamard(d)
        q, k = q @ hm * (8.0 / d), k @ hm / 8.0
    up = U["f16"] if quant else U[dtype]
    ok = A.seen(lq, lk, window)
    tol = np.zeros((lq, h))
    for i in range(h):
        qq, kk, vv = q[:, i], k[:, i * kv // h], v[:, i * kv // h]
        s = np.where(ok, scale * (qq @ kk.T), -np.inf)
        top = s.max(-1, keepdims=True, initial=-np.inf)
        w = np.where(ok, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
        total = w.sum(-1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
        vn = np.linalg.norm(vv, axis=-1)[None]
        on = np.linalg.norm(out[:, i], axis=-1)[:, None]
        e = scale * np.sqrt(2.0) * u * np.sqrt((qq * qq) @ (kk * kk).T)
        e = e + 2.0**-20 * (1.0 + scale * (np.abs(qq) @ np.abs(kk).T))
        each = (w * e * (vn + on)) ** 2 + (w * vn) ** 2 * (up**2 + u**2)
        if quant or dtype == "f16":
            each = each + (2.0**-25 * (w * vn).max(-1, keepdims=True, initial=0.0)) ** 2 * ok
        tol[:, i] = 4.0 * np.sqrt(each.sum(-1)) + 2.0**-20 * (w * vn).sum(-1)
        tol[:, i] += U[dtype] * (on[:, 0] + tol[:, i]) + (2.0**-25 if dtype == "f16" else 1e-38) * d**0.5
    return out, tol


def rows_off(got, want, tol):
    """The error of every row over its bound."""
    assert got.shape == want.shape
    return np.linalg.norm(got - want, axis=-1) / tol


def assert_rows(got, want, tol, what=""):
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    off = rows_off(got, want, tol)
    worst = float(off.max()) if off.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of the bound at row {np.unravel_index(np.argmax(off), off.shape)}"
