"""Norms and rotation, their gradients, and the 4-bit cache's rows, in plain
NumPy and float64, from the definitions.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): the product path never
imports this module.
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E5M3 = np.array([f / 8 * 2.0 ** -14 for f in range(8)] + [(1 + f / 8) * 2.0 ** (e - 15) for e in range(1, 31) for f in range(8)])


def norm(x, w, eps):
    """n(x) over the last axis (w None: x)."""
    x = np.asarray(x, np.float64)
    return x if w is None else x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(w, np.float64)


def pairs(rot, inter):
    """Indices of the pairs' first and second elements."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def rotate(x, cos, sin, inter, dtype=np.float64):
    """x [.., H, d] by the angles of cos, sin [.., rot / 2]; with float32 each
    product and sum is rounded by itself."""
    x = np.asarray(x, dtype)
    a, b = pairs(2 * cos.shape[-1], inter)
    c, s = np.asarray(cos, dtype)[..., None, :], np.asarray(sin, dtype)[..., None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def reach(x, cos, sin, inter):
    """|a c| + |b s| of each output element of rotate: what its rounding errors go by."""
    x = np.abs(np.asarray(x, np.float64))
    return rotate_abs(x, np.abs(cos), np.abs(sin), inter)


def rotate_abs(x, cos, sin, inter):
    a, b = pairs(2 * cos.shape[-1], inter)
    c, s = np.asarray(cos, np.float64)[..., None, :], np.asarray(sin, np.float64)[..., None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c + x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def grads(dy, x, cos, sin, w, eps, inter):
    """(dx, dw) of rotate(norm(x)); dw None without weights."""
    u = rotate(dy, cos, -np.asarray(sin), inter)
    if w is None:
        return u, None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    t = u * w
    dx = r * (t - x * r * r * np.mean(t * x, -1, keepdims=True))
    return dx, np.sum((u * x * r).reshape(-1, x.shape[-1]), 0)


def nearest(x, values):
    """Index of the nearest of ascending values to each x >= 0, ties to the even index."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    below, above = x - values[hi - 1], values[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x):
    """Rows [.., d] -> codes 0 .. 15 [.., d] and scale bytes [.., d / 32]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (-1, 32))
    most = np.max(np.abs(g), -1)
    bad = ~np.isfinite(most)
    s = np.where(bad, 0xFC, nearest(np.where(bad, 0, most) / 6, E5M3)).astype(np.uint8)
    scale = np.where(bad, 0.0, E5M3[np.minimum(s, len(E5M3) - 1)])[..., None]
    q = np.where(scale > 0, np.where(np.isfinite(g), g, 0) / np.where(scale > 0, scale, 1), 0)
    c = nearest(np.abs(q), E2M1) + 8 * (q < 0)
    return c.reshape(x.shape).astype(np.uint8), s


def place(d):
    """Nibble of each element of a row."""
    i = np.arange(d)
    return i % 32 // 4 * (d // 32) * 4 + i // 32 * 4 + i % 4


def pack(codes):
    """Codes [.., d] -> bytes [.., d / 2]."""
    d = codes.shape[-1]
    n = np.empty_like(codes)
    n[..., place(d)] = codes
    return n[..., 0::2] | n[..., 1::2] << 4


def scales(b):
    b = np.asarray(b)
    return np.where(b < 0xF8, E5M3[np.minimum(b, len(E5M3) - 1)], np.nan)


def unpack(rows, b):
    """What bytes [.., d / 2] and scale bytes [.., d / 32] stand for."""
    d = 2 * rows.shape[-1]
    n = np.stack([rows & 15, rows >> 4], -1).reshape(rows.shape[:-1] + (d,))[..., place(d)]
    v = np.where(n >= 8, -1.0, 1.0) * E2M1[n & 7]
    return v * np.repeat(scales(b), 32, -1)
