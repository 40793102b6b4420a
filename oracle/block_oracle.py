"""Operators around a block's weights in numpy float64, from the definitions: the product with
a weight matrix (bias, activation, residual), the RMS norm of the residual stream with its 8-bit
form, the embedding, the norm of all gradients, and the gradients.

Matrices are [rows, columns].
"""

from __future__ import annotations

import numpy as np

GELU_A, GELU_B = np.sqrt(2.0 / np.pi), 0.044715
E4M3_MAX = 448.0


# ------------------------------------------------------------ linear
def act(z, kind):
    if kind == "relu2":
        return np.where(z <= 0, 0.0, z * z)
    if kind == "gelu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-2.0 * GELU_A * (z + GELU_B * z ** 3)))
    return z


def slope(z, kind):
    if kind == "relu2":
        return np.where(z <= 0, 0.0, 2.0 * z)
    if kind == "gelu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-2.0 * GELU_A * (z + GELU_B * z ** 3)))
        return s + 2.0 * z * s * (1.0 - s) * GELU_A * (1.0 + 3.0 * GELU_B * z * z)
    return np.ones_like(z)


def linear(x, w, bias=None, kind=None, residual=None):
    """(out, z): z = x w^T + bias, out = act(z) + residual."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act(z, kind)
    return (y if residual is None else y + residual), z


def linear_backward(dout, x, w, kind=None, z=None):
    """(dx, dw, dbias) with the activation's slope taken at z."""
    dz = dout if kind is None else dout * slope(z, kind)
    return dz @ w, dz.T @ x, dz.sum(0)


# ------------------------------------------------------------ RMS norm
def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """(y, h): h = x + residual, y = h (mean h^2 + eps)^-1/2 weight."""
    h = x if residual is None else x + residual
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return (y if weight is None else y * weight), h


def rms_norm_backward(dout, h, weight=None, dresidual=None, eps=1e-6):
    """(dx, dweight)."""
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    n = h * r
    g = dout if weight is None else dout * weight
    dx = r * (g - n * np.mean(g * n, axis=1, keepdims=True))
    if dresidual is not None:
        dx = dx + dresidual
    return dx, (dout * n).sum(0)


def e4m3(v):
    """The nearest e4m3 value (ties to even) of |v| <= 464: 3 bits behind the point from 2^-6 on,
    multiples of 2^-9 below."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = np.exp2(e - 3)
    return np.round(v / step) * step


def group_scales(y, group):
    """The least power of two for each group that brings its largest |y| to 448 or less, and at
    least 2^-126; 1 where all is 0, NaN where something is not finite.  [rows, groups]."""
    rows, cols = y.shape
    width = group or cols
    out = np.empty((rows, -(-cols // width)))
    for g in range(out.shape[1]):
        top = np.abs(y[:, g * width:(g + 1) * width]).max(axis=1)
        for i, t in enumerate(top):
            if not np.isfinite(t):
                out[i, g] = np.nan
            elif t == 0:
                out[i, g] = 1.0
            else:
                e = -126
                while t > E4M3_MAX * 2.0 ** e:
                    e += 1
                out[i, g] = 2.0 ** e
    return out


def spread(scales, cols, group):
    """Scales at every column."""
    return np.repeat(scales, group or cols, axis=1)[:, :cols]


# ------------------------------------------------------------ embedding
def embedding(ids, table, scale=1.0):
    good = (ids >= 0) & (ids < len(table))
    out = scale * table[np.where(good, ids, 0)]
    out[~good] = np.nan
    return out


def embedding_backward(dout, ids, rows, scale=1.0):
    out = np.zeros((rows, dout.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < rows:
            out[v] += dout[t]
    return scale * out


# ------------------------------------------------------------ clipping
def grad_norm(grads):
    return np.sqrt(sum(float(np.sum(g.astype(np.float64) ** 2)) for g in grads))


def clip_factor(norm, max_norm, eps=1e-6):
    return min(1.0, max_norm / (norm + eps))
