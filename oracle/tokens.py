"""fp64 definitions of the token operators: layer norm, rotary positions with
several axes, attention over packed sequences, and their gradients.

Plain numpy over unsharded arrays, independent of the library.  The
transformers of "Technical summary: ShardTensor", section 4 ("Results and
benchmarks") run these over the sharded grids; the operators themselves are the
textbook ones.
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """x [..., C] -> (y, mean [...], rstd [...])."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean, rstd


def layer_norm_backward(x, dy, gamma=None, eps=1e-5):
    """(dx, dgamma, dbeta)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    _, mean, rstd = layer_norm(x, eps=eps)
    xhat = (x - mean[..., None]) * rstd[..., None]
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - xhat * (g * xhat).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (dy * xhat).sum(axes), dy.sum(axes)


def rope(x, positions, axis_dims, base=10000.0, pairs="halves", inverse=False, rotated_heads=None):
    """x [T, H, D], positions [T, axes] -> rotated copy."""
    out = np.array(x, np.float64)
    src = np.asarray(x, np.float64)
    r = out.shape[1] if rotated_heads is None else rotated_heads
    lo = 0
    for a, d in enumerate(axis_dims):
        for i in range(d // 2):
            m, n = (lo + i, lo + d // 2 + i) if pairs == "halves" else (lo + 2 * i, lo + 2 * i + 1)
            angle = np.asarray(positions, np.float64)[:, a] * base ** (-2.0 * i / d) * (-1.0 if inverse else 1.0)
            c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
            u, v = src[:, :r, m], src[:, :r, n]
            out[:, :r, m], out[:, :r, n] = u * c - v * s, u * s + v * c
        lo += d
    return out


def seen(lq, lk, causal):
    """[lq, lk] mask of the keys each query sees."""
    if not causal:
        return np.ones((lq, lk), bool)
    return np.arange(lk)[None, :] <= np.arange(lq)[:, None] + lk - lq


def attention_one(q, k, v, scale, causal, dout=None):
    """One sequence and head: q [lq, D], k, v [lk, D].  Returns a dict of the
    outputs, the weights p, and with dout the gradients and ds."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    s = scale * (q @ k.T)
    mask = seen(len(q), len(k), causal)
    s = np.where(mask, s, -np.inf)
    with np.errstate(all="ignore"):
        m = s.max(1, keepdims=True) if s.shape[1] else np.full((len(q), 1), -np.inf)
        e = np.where(mask, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
        l = e.sum(1, keepdims=True)
        p = np.where(l > 0, e / np.where(l > 0, l, 1.0), 0.0)
        lse = np.where(l[:, 0] > 0, np.where(np.isfinite(m), m, 0.0)[:, 0] + np.log(l[:, 0]), -np.inf)
    r = {"out": p @ v, "lse": lse, "p": p}
    if dout is not None:
        dout = np.asarray(dout, np.float64)
        dp = dout @ v.T
        ds = p * (dp - (dout * r["out"]).sum(1, keepdims=True))
        r.update(ds=ds, dp=dp, dq=scale * ds @ k, dk=scale * ds.T @ q, dv=p.T @ dout)
    return r


def attention(q, k, v, q_lens, k_lens, scale, causal, dout=None):
    """Packed q [Tq, H, D], k, v [Tk, Hkv, D].  Returns out, lse [Tq, H] and with
    dout also dq, dk, dv (dk, dv summed over the heads that share them)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    group = q.shape[1] // k.shape[1]
    r = {"out": np.zeros_like(q), "lse": np.zeros(q.shape[:2])}
    if dout is not None:
        r.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    i = j = 0
    for lq, lk in zip(q_lens, k_lens):
        rows, keys = slice(i, i + lq), slice(j, j + lk)
        for h in range(q.shape[1]):
            one = attention_one(q[rows, h], k[keys, h // group], v[keys, h // group], scale, causal,
                                None if dout is None else np.asarray(dout)[rows, h])
            r["out"][rows, h], r["lse"][rows, h] = one["out"], one["lse"]
            if dout is not None:
                r["dq"][rows, h] = one["dq"]
                r["dk"][keys, h // group] += one["dk"]
                r["dv"][keys, h // group] += one["dv"]
        i, j = i + lq, j + lk
    return r


def attention_bounds(q, k, v, q_lens, k_lens, scale, causal, dout):
    """Absolute values that rounding errors of the outputs scale with, each laid
    out as its output: for out and dv the weights times the absolute values
    they multiply; for dq and dk, |ds| + p (|dout| |out|) times the absolute
    values of the other factor, times scale; and the largest scale * sum |q||k|."""
    q, k, v, dout = (np.asarray(a, np.float64) for a in (q, k, v, dout))
    group = q.shape[1] // k.shape[1]
    b = {"out": np.zeros_like(q), "dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "score": 0.0}
    i = j = 0
    for lq, lk in zip(q_lens, k_lens):
        rows, keys = slice(i, i + lq), slice(j, j + lk)
        for h in range(q.shape[1]):
            g = h // group
            qq, kk, vv, gg = q[rows, h], k[keys, g], v[keys, g], dout[rows, h]
            one = attention_one(qq, kk, vv, scale, causal, gg)
            if lq and lk:
                b["score"] = max(b["score"], scale * float((np.abs(qq) @ np.abs(kk).T).max()))
            w = np.abs(one["ds"]) + one["p"] * (np.abs(gg) @ np.abs(vv).T + (np.abs(gg) * np.abs(one["out"])).sum(1, keepdims=True))
            b["out"][rows, h] = one["p"] @ np.abs(vv)
            b["dq"][rows, h] = scale * w @ np.abs(kk)
            b["dk"][keys, g] += scale * w.T @ np.abs(qq)
            b["dv"][keys, g] += one["p"].T @ np.abs(gg)
        i, j = i + lq, j + lk
    return b
