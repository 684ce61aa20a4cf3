"""fp64 definitions of the MLP branch's operators: matrix product with bias,
activation and residual, root-mean-square norm with the residual's addition,
the 8-bit form of activations, and the gradients.

Plain numpy, independent of the library.
"""
from __future__ import annotations

import numpy as np
from scipy.special import ndtr


def activate(z, act):
    z = np.asarray(z, np.float64)
    if act == "relu":
        return np.maximum(z, 0)
    if act == "gelu":
        return z * ndtr(z)
    if act == "silu":
        return z / (1 + np.exp(-z))
    return z


def slope(z, act):
    z = np.asarray(z, np.float64)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if act == "silu":
        t = 1 / (1 + np.exp(-z))
        return t * (1 + z * (1 - t))
    return np.ones_like(z)


def linear(x, w, bias=None, act="none", residual=None):
    """(y, pre): act(x w^T + bias) + residual and x w^T + bias."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = activate(z, act)
    return (y if residual is None else y + np.asarray(residual, np.float64)), z


def linear_backward(x, w, dy, act="none", pre=None):
    """(dx, dw, dbias)."""
    p = np.asarray(dy, np.float64)
    if act != "none":
        p = p * slope(pre, act)
    return p @ np.asarray(w, np.float64), p.T @ np.asarray(x, np.float64), p.sum(0)


def rms_norm(s, gamma=None, eps=1e-6):
    """(y, rstd) of the sum s [rows, channels]."""
    s = np.asarray(s, np.float64)
    rstd = 1 / np.sqrt((s * s).mean(-1) + eps)
    y = s * rstd[:, None]
    return (y if gamma is None else y * np.asarray(gamma, np.float64)), rstd


def rms_norm_backward(s, dy, dtotal=None, gamma=None, rstd=None, eps=1e-6):
    """(dx, dgamma); rstd: of the sum before it was kept in fewer bits, if not s's own."""
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    if rstd is None:
        rstd = rms_norm(s, eps=eps)[1]
    r = np.asarray(rstd, np.float64)[:, None]
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    xh = s * r
    dx = r * (g - xh * (g * xh).mean(-1, keepdims=True))
    return (dx if dtotal is None else dx + np.asarray(dtotal, np.float64)), (dy * xh).sum(0)


def e4m3_table():
    """Values of the 256 codes: bias 7, subnormals of 2^-9, 0x7F and 0xFF NaN, no infinity."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v[c] = np.nan if c & 127 == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        if c > 127:
            v[c] = -v[c]
    return v


def mx8_values(codes, scales, channels):
    """Values of codes [rows, >= channels] and scale bytes (0: 2^-127, 255: NaN)."""
    codes, scales = np.asarray(codes), np.asarray(scales).astype(np.int64)
    block = np.arange(channels) // 32
    k = scales[:, block]
    f = np.where(k == 255, np.nan, 2.0 ** (np.minimum(k, 254) - 127.0))
    return e4m3_table()[codes[:, :channels]] * f


def mx8_store(x):
    """(codes, scales) of x [rows, channels]: per block of 32 channels the smallest
    power 2^k (k of -126 .. 127) with max |x| <= 448 * 2^k over the finite values,
    the nearest of the code values, ties to the even code; NaN code else."""
    x = np.asarray(x, np.float64)
    rows, c = x.shape
    finite = np.isfinite(x)
    a = np.where(finite, np.abs(x), 0.0)
    blocks = -(-c // 32)
    top = np.pad(a, ((0, 0), (0, -c % 32))).reshape(rows, blocks, 32).max(-1)
    k = np.full((rows, blocks), -126)
    for p in range(-126, 127):
        k = np.where(top > 448 * 2.0 ** p, p + 1, k)
    table = e4m3_table()[:127]                            # 0 .. 448, ascending with the code
    u = a * 2.0 ** -k[:, np.arange(c) // 32].astype(np.float64)
    hi = np.minimum(np.searchsorted(table, u), 126)
    lo = np.maximum(hi - 1, 0)
    down, up = u - table[lo], table[hi] - u
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(finite, code | np.where(np.signbit(x), 128, 0), 127)
    return code.astype(np.uint8), (k + 127).astype(np.uint8)
