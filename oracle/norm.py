"""Residual addition with a root-mean-square norm, and its backward pass, from their definitions in
64 bits (numpy)."""
import numpy as np

E4M3_MAX, SCALE_MIN = 448.0, 2.0 ** -100


def forward(x, residual, weight, eps):
    """(h, rstd, y) for rows x cols arrays (residual, weight: or None)."""
    h = x.astype(np.float64) if residual is None else x.astype(np.float64) + residual.astype(np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    y = h * rstd[:, None]
    return h, rstd, y if weight is None else y * weight.astype(np.float64)


def scales(y, group):
    """One scale per row and group of columns (group 0: the row): [rows, groups]."""
    cols = y.shape[1]
    step = group or cols
    return np.stack([np.maximum(np.abs(y[:, c:c + step]).max(axis=1) / E4M3_MAX, SCALE_MIN)
                     for c in range(0, cols, step)], axis=1)


def spread(s, group, cols):
    """Scales [rows, groups] as one per element."""
    return np.repeat(s, group or cols, axis=1)[:, :cols]


def backward(dy, h, weight, rstd, dres):
    """(dx, dweight)."""
    dy, h, s = dy.astype(np.float64), h.astype(np.float64), rstd.astype(np.float64)[:, None]
    n = h * s
    g = dy if weight is None else dy * weight.astype(np.float64)
    dx = s * (g - n * (g * n).mean(axis=1, keepdims=True))
    return dx if dres is None else dx + dres.astype(np.float64), (dy * n).sum(axis=0)
