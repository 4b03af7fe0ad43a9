"""The bound that attention results are held to, against the FP64 oracle.

Let w be the exact weights, A = sum w|v| and o = sum w v (oracle: spread, out), R the largest scale * sum_d |q_d k_d| of a
row (reach).  An error of at most e in every score changes o by at most (e^e - 1)(A + |o|); weights rounded to a type of
unit roundoff u_p change it by u_p A, values rounded by u_v A; the result rounds by u_o |o|.
  e: fp32 sums of D products, D 2^-24 R at the most; the scaled score's own roundings, the exponent's and ex2's (2^-22
     of weights up to the score range) 2^-20 (1 + R) in all; over a quantised cache q and the keys round to fp16 in the
     rotated basis: 2 * 2^-11 R' with R' of the rotated rows.
  The sum of the weights is fp32: 2^-20 A.
Weights below fp16's normal range are off by 2^-25 of the reference weight at the most, n of them by n 2^-25 max|v|.
Over a quantised cache the bound holds in the rotated basis; rotating back sums D entries' errors times 8 / D.
"""
import numpy as np

from oracle import attention_oracle as A

U = {"bf16": 2.0**-8, "f16": 2.0**-11}  # one rounding to nearest, half an ulp, relative


def bound(q, k, v, window, scale, dtype, fmt):
    """(out, tolerance) of one sequence; q, k, v in 64 bits as the library is given them (k, v read back for int8/int4)."""
    d = q.shape[-1]
    quant = fmt in A.TOP
    if quant:
        hm = A.hadamard(d)
        q, k, v = q @ hm * (8.0 / d), k @ hm / 8.0, v @ hm / 8.0
    out, spread, reach = A.attention(q, k, v, window, scale)
    e = reach * (d * 2.0**-24 + 2.0**-20 + (2 * 2.0**-11 if quant else 0.0)) + 2.0**-20
    up = U["f16"] if quant else U[dtype]
    tol = np.expm1(e)[..., None] * (spread + np.abs(out)) + (up + (2.0**-11 if quant else 0.0) + 2.0**-20) * spread
    if quant or dtype == "f16":
        n = k.shape[0]
        tol = tol + n * 2.0**-25 * (np.abs(v).max() if v.size else 0.0)
    if quant:
        out = out @ hm * (8.0 / d)
        tol = np.repeat(tol.sum(-1, keepdims=True) * (8.0 / d), d, -1)
    # the final rounding, and the smallest step of the type
    return out, tol * (1 + 2 * U[dtype]) + U[dtype] * np.abs(out) + (2.0**-25 if dtype == "f16" else 1e-30)


def assert_close(got, want, tol, what=""):
    assert got.shape == want.shape
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    err = np.abs(got - want)
    worst = float((err / tol).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} of the bound at {np.unravel_index(np.argmax(err / tol), err.shape)}"
