"""Attention path in numpy float64: norm and rotation of the query and key heads, causal
attention over packed sequences, and the gradients of both, from the definitions.

Arrays are [tokens, heads, head_dim].  Only visible (query, key) pairs enter a sum, so
that Inf or NaN elsewhere leaves a row alone.
"""

from __future__ import annotations

import numpy as np


def pairs(rot_dim, interleaved):
    i = np.arange(rot_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)


def rotate(x, cos, sin, positions, interleaved):
    """x with the pairs of its first 2 * cos.shape[1] elements rotated by rows `positions`."""
    a, b = pairs(2 * cos.shape[1], interleaved)
    c, s = cos[positions][:, None, :], sin[positions][:, None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, weight, cos, sin, positions, *, norm=True, eps=1e-6, interleaved=False):
    n = x
    if norm:
        n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        if weight is not None:
            n = n * weight
    return rotate(n, cos, sin, positions, interleaved)


def norm_rope_backward(dy, x, weight, cos, sin, positions, *, norm=True, eps=1e-6,
                       interleaved=False):
    """(dx, dweight); dweight is None without a norm."""
    g = rotate(dy, cos, -sin, positions, interleaved)
    if not norm:
        return g, None
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    h = x * r
    dw = np.sum(g * h, axis=(0, 1))
    gw = g if weight is None else g * weight
    return r * (gw - h * np.mean(gw * h, axis=-1, keepdims=True)), dw


def spans(cu_seqlens, tokens):
    """(begin, end) of each non-empty sequence."""
    cu = [0, tokens] if cu_seqlens is None else list(cu_seqlens)
    return [(a, b) for a, b in zip(cu[:-1], cu[1:]) if b > a]


def _hide(x, visible, value=0.0):
    return np.where(visible, x, value)


def _sum(weights, rows, visible):
    """weights @ rows over the visible pairs only (visible pairs may hold Inf or NaN)."""
    if np.isfinite(rows).all() and np.isfinite(weights).all():
        return _hide(weights, visible) @ rows
    out = np.empty((weights.shape[0], rows.shape[1]))
    for i in range(weights.shape[0]):
        out[i] = weights[i, visible[i]] @ rows[visible[i]]
    return out


def attention(q, k, v, cu_seqlens=None, scale=None):
    """(out, lse [heads, tokens]); tokens outside every sequence get 0 and -inf."""
    t, hq, d = q.shape
    group = hq // k.shape[1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out = np.zeros((t, hq, v.shape[2]))
    lse = np.full((hq, t), -np.inf)
    for a, b in spans(cu_seqlens, t):
        vis = np.tril(np.ones((b - a, b - a), dtype=bool))
        for h in range(hq):
            s = _hide(scale * (q[a:b, h] @ k[a:b, h // group].T), vis, -np.inf)
            m = s.max(axis=1)
            p = np.exp(s - m[:, None])
            l = p.sum(axis=1)
            lse[h, a:b] = m + np.log(l)
            out[a:b, h] = _sum(p / l[:, None], v[a:b, h // group], vis)
    return out, lse


def attention_backward(dout, q, k, v, out, lse, cu_seqlens=None, scale=None):
    """(dq, dk, dv) with delta = dout . out of the given out, p = exp(s - the given lse)."""
    t, hq, d = q.shape
    group = hq // k.shape[1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, b in spans(cu_seqlens, t):
        vis = np.tril(np.ones((b - a, b - a), dtype=bool))
        for h in range(hq):
            g = h // group
            qq, kk, vv, do = q[a:b, h], k[a:b, g], v[a:b, g], dout[a:b, h]
            p = np.exp(_hide(scale * (qq @ kk.T), vis, -np.inf) - lse[h, a:b, None])
            delta = np.sum(do * out[a:b, h], axis=1, keepdims=True)
            ds = _hide(p * (do @ vv.T - delta), vis)
            dq[a:b, h] = scale * _sum(ds, kk, vis)
            dk[a:b, g] += scale * _sum(ds.T, qq, vis.T)
            dv[a:b, g] += _sum(p.T, do, vis.T)
    return dq, dk, dv
