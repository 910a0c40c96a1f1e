"""Plain binary64 forms of the operators around a block's linears: layer norm and low-rank adapters, with their
gradients.  numpy only; shares no code with the GPU path."""
import numpy as np


def layer_norm(x, w, b, eps):
    """(y, mean, rstd, xhat) of the rows of x; w and b may be None."""
    mean = x.mean(1, keepdims=True)
    var = ((x - mean) ** 2).mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(var + eps)
    xhat = (x - mean) * rstd
    y = xhat if w is None else xhat * w
    return (y if b is None else y + b), mean, rstd, xhat


def layer_norm_grads(dy, xhat, rstd, w):
    """(dx, dw, db)."""
    g = dy if w is None else dy * w
    dx = rstd * (g - g.mean(1, keepdims=True) - xhat * (g * xhat).mean(1, keepdims=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def lora(base, x, a, b, index, scales):
    """(y, h): y (T, N), h (T, R) the inner products times their scale (0 without an adapter)."""
    y, h = base.copy(), np.zeros((x.shape[0], a.shape[1]))
    for i in range(a.shape[0]):
        rows = np.flatnonzero(index == i)
        h[rows] = scales[i] * (x[rows] @ a[i].T)
        y[rows] += h[rows] @ b[i].T
    return y, h


def lora_grads(dy, x, a, b, index, scales, h):
    """(dx, da, db, g)."""
    dx, g = np.zeros_like(x), np.zeros_like(h)
    da, db = np.zeros_like(a), np.zeros_like(b)
    for i in range(a.shape[0]):
        rows = np.flatnonzero(index == i)
        g[rows] = scales[i] * (dy[rows] @ b[i])
        dx[rows] = g[rows] @ a[i]
        da[i] = g[rows].T @ x[rows]
        db[i] = dy[rows].T @ h[rows]
    return dx, da, db, g
