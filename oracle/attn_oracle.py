"""Plain FP64 oracle for rotary positions, the paged KV cache and attention.

TEST INFRASTRUCTURE ONLY -- never called by the product path.

The formulas are those of include/wal.h ("between the q, k, v products and the
o product"); the model cards give a KV cache and contexts but no layouts, so
the readings are the library's own.  Everything is float64 on numpy arrays,
one sequence and one head at a time.
"""
from __future__ import annotations

import math

import numpy as np

FLT_MIN = float(np.finfo(np.float32).tiny)
QMAX = {"int8": 127.0, "e4m3": 448.0}


def rope_freqs(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, slow=1.0, fast=32.0):
    """Radians a position of each pair, and the factor on the result."""
    f = np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        g = np.clip((original_len * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        return (1 - g) * f / factor + g * f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, pos, freqs, mscale=1.0, layout="half"):
    """x [T, heads, D] at positions pos [T]; the first 2 * len(freqs) columns turn."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    n = len(freqs)
    for i, f in enumerate(freqs):
        lo, hi = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        a = (np.asarray(pos, np.float64) * f)[:, None]
        y[..., lo] = mscale * (x[..., lo] * np.cos(a) - x[..., hi] * np.sin(a))
        y[..., hi] = mscale * (x[..., hi] * np.cos(a) + x[..., lo] * np.sin(a))
    return y


def e4m3_values(bits):
    """Values of finite e4m3 codes."""
    b = np.asarray(bits).astype(np.int64) & 0xFF
    e, m = (b >> 3) & 15, b & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    return np.where(b & 0x80, -mag, mag)


def scales(x, typ):
    """Scale of every row (last axis) of x."""
    return np.maximum(np.abs(x).max(-1) / QMAX[typ], FLT_MIN)


def step(y, typ):
    """Distance of neighbouring code values around y (in units of the scale)."""
    if typ == "int8":
        return np.ones_like(y)
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)


def attend(q, k, v, scale, group):
    """One sequence: q [n, heads, D] the last n of its tokens, k and v
    [len, kv_heads, D].  Returns (o, a): the outputs [n, heads, D] and
    a = sum_j w_j |v_j|, the size that rounding errors of the weights act on."""
    n, heads, D = q.shape
    L = k.shape[0]
    o, a = np.zeros((n, heads, D)), np.zeros((n, heads, D))
    if L == 0:
        return o, a
    sees = np.arange(L) <= (L - n + np.arange(n))[:, None]
    some = sees.any(1)
    for h in range(heads):
        s = np.where(sees, q[:, h] @ k[:, h // group].T * scale, -np.inf)[some]
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        o[some, h] = w @ v[:, h // group]
        a[some, h] = w @ np.abs(v[:, h // group])
    return o, a
