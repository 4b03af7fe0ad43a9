"""FP64 CPU oracle of the rotary, cache and attention calls.

Plain numpy from the definitions in include/exl3.h; shares no code with the CUDA path.  Rows are [tokens, heads,
head_dim].  Where the library's result is a rounding of fp32 steps that are themselves part of the definition (the
quantised rows), the same steps are done in numpy's fp32.
"""
import math

import numpy as np

TOP = {"int8": 127, "int4": 7}
BIAS = {"int8": 128, "int4": 8}


def phases(rot_dim, base=10000.0, scaling="plain", factor=1.0, fast=32.0, slow=1.0, original_len=4096.0):
    """(frequencies in radians a position, amplitude)."""
    i = np.arange(rot_dim // 2)
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        g = np.clip((original_len * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * (g + (1 - g) / factor)
    return f, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rope(x, positions, phase_words, layout, amplitude):
    """x [T, H, D] rotated; phase_words: unsigned 64-bit turns a position."""
    t = np.array([[(int(p) * int(w)) % 2**64 / 2.0**64 for w in phase_words] for p in positions])
    c, s = np.cos(2 * math.pi * t)[:, None], np.sin(2 * math.pi * t)[:, None]
    n = len(phase_words)
    y = np.array(x, dtype=np.float64)
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    a, b = x[..., first], x[..., second]
    y[..., first] = amplitude * (a * c - b * s)
    y[..., second] = amplitude * (b * c + a * s)
    return y


def hadamard(d):
    return np.array([[-1.0 if bin(i & j).count("1") % 2 else 1.0 for j in range(d)] for i in range(d)])


def quantise(x, fmt):
    """(codes, scales) of rows x [..., D] (values exact in fp32), by the format's own fp32 steps."""
    y = np.asarray(x, dtype=np.float32)
    d, s = y.shape[-1], 1
    while s < d:
        p = y.reshape(*y.shape[:-1], d // (2 * s), 2, s)
        with np.errstate(invalid="ignore"):
            y = np.stack([p[..., 0, :] + p[..., 1, :], p[..., 0, :] - p[..., 1, :]], axis=-2).reshape(y.shape)
        s *= 2
    y = y * np.float32(0.125)
    fine = np.isfinite(y).all(-1, keepdims=True)
    y = np.where(fine, y, np.float32(0))
    top = np.abs(y).max(-1, keepdims=True)
    raw = (top * np.float32(1.0 / TOP[fmt])).astype(np.float32)
    up = ((raw.view(np.uint32) + np.uint32(0xFFFF)) & np.uint32(0xFFFF0000)).view(np.float32)
    scale = np.where(top == 0, np.float32(1), np.maximum(up, np.float32(2.0**-100)))
    codes = np.clip(np.rint(y * (np.float32(1) / scale)), -TOP[fmt], TOP[fmt]).astype(np.int64)
    return np.where(fine, codes, 0), np.where(fine, scale, np.float32(np.nan))[..., 0]


def stored(codes, fmt):
    """Codes as the cache holds them (bytes)."""
    c = (codes + BIAS[fmt]).astype(np.uint8)
    return c if fmt == "int8" else (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def codes_of(data, fmt):
    if fmt == "int8":
        return data.astype(np.int64) - 128
    out = np.empty(data.shape[:-1] + (2 * data.shape[-1],), dtype=np.int64)
    out[..., 0::2] = (data & 15).astype(np.int64) - 8
    out[..., 1::2] = (data >> 4).astype(np.int64) - 8
    return out


def read_back(codes, scales):
    d = codes.shape[-1]
    return (codes.astype(np.float64) @ hadamard(d)) * (scales.astype(np.float64)[..., None] * (8.0 / d))


def seen(q_len, kv_len, window):
    """[q_len, kv_len]: which keys the sequence's last q_len tokens see."""
    pos = kv_len - q_len + np.arange(q_len)[:, None]
    j = np.arange(kv_len)[None, :]
    ok = j <= pos
    return ok & (j > pos - window) if window else ok


def attention(q, k, v, window=0, scale=None):
    """One sequence: q [Lq, H, D], k and v [Lk, KV, D] -> (out, spread, reach).

    spread [Lq, H, D]: sum_j w_j |v_j| / sum_j w_j; reach [Lq, H]: scale * max_j sum_d |q_d k_jd| over the keys seen
    (what rounding errors of weights, values and scores are bounded by)."""
    lq, h, d = q.shape
    lk, kv, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    out, spread, reach = np.zeros((lq, h, d)), np.zeros((lq, h, d)), np.zeros((lq, h))
    ok = seen(lq, lk, window)
    for i in range(h):
        kk, vv = k[:, i * kv // h], v[:, i * kv // h]
        s = np.where(ok, scale * (q[:, i] @ kk.T), -np.inf)
        big = np.where(ok, scale * (np.abs(q[:, i]) @ np.abs(kk).T), 0.0)
        top = s.max(-1, keepdims=True, initial=-np.inf)
        w = np.where(ok, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
        total = w.sum(-1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
        # a key that is not seen takes no part, whatever it holds
        vz = np.where(ok.any(0)[:, None], vv, 0.0)
        out[:, i], spread[:, i] = w @ vz, w @ np.abs(vz)
        reach[:, i] = big.max(-1, initial=0.0)
    return out, spread, reach
