"""Inputs and error bounds shared by the layer norm's and the adapters' tests.

u = 2^-24 is half a step of binary32; a sum of terms t added in any order with at most d roundings on a term's way is
off by at most d u sum|t| (1 + d u) -- the bounds below take 1.01 for that last factor.  A matrix instruction's sums
may be truncated rather than rounded: twice that."""
import numpy as np
import torch

from oracle import block

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def draw(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std + mean).to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def half_step(ref, dtype):
    """Half a step of `dtype` at |ref|, or of its subnormals."""
    info = torch.finfo(dtype)
    return np.maximum(np.abs(ref) * (info.eps / 2), info.smallest_normal * info.eps / 2)


def close(got, ref, err, what):
    """got within err (before rounding) plus half a step of its type."""
    ref = np.asarray(ref)
    tol = 1.01 * err + half_step(np.abs(ref) + 1.01 * err, got.dtype)
    bad = ~(np.abs(np64(got) - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.nanmax(np.abs(np64(got) - ref) / np.maximum(tol, 1e-300))))


def norm_bounds(x, w, b, eps, rows, cols):
    """Of layer_norm's binary64 (y, mean, rstd, xhat): the errors a binary32 evaluation can have, as a dict."""
    y, mean, rstd, xhat = block.layer_norm(x, w, b, eps)
    # roundings on an element's way into a row's sum: at most 32 in a thread (cols / 1024 in the widest rows), 6 in the
    # wave, 16 over the waves, and the division
    d = 64 + cols / 1024
    sd = np.sqrt(((x - mean) ** 2).mean(1, keepdims=True))
    d_mean = d * U * np.abs(x).mean(1, keepdims=True)
    # (x - mean)^2: an error of d_mean in each difference, then its own rounding twice
    d_var = 2 * sd * d_mean + d_mean ** 2 + (d + 4) * U * sd ** 2
    rel = 0.5 * d_var * rstd ** 2 * (1 + d_var * rstd ** 2) + 4 * U
    d_xhat = np.abs(xhat) * (rel + 3 * U) + rstd * d_mean * (1 + rel)
    aw = 1.0 if w is None else np.abs(w)
    d_y = aw * d_xhat + 2 * U * np.abs(y) + (0 if b is None else 2 * U * np.abs(b))
    return dict(y=y, mean=mean, rstd=rstd, xhat=xhat, rel=rel, d=d, d_xhat=d_xhat, d_y=d_y)


def norm_grad_bounds(n, dy, w, rows, cols):
    """((dx, dw, db), their errors)."""
    refs = block.layer_norm_grads(dy, n["xhat"], n["rstd"], w)
    g = np.abs(dy if w is None else dy * w)
    xh = np.abs(n["xhat"])
    gm = (dy if w is None else dy * w)
    m0, m1 = np.abs(gm.mean(1, keepdims=True)), np.abs((gm * n["xhat"]).mean(1, keepdims=True))
    d0 = (n["d"] + 2) * U * g.mean(1, keepdims=True)
    d1 = (n["d"] + 3) * U * (g * xh).mean(1, keepdims=True) + (g * n["d_xhat"]).mean(1, keepdims=True)
    d_dx = n["rstd"] * (1 + n["rel"]) * (4 * U * (g + m0 + xh * m1) + d0 + (xh + n["d_xhat"]) * d1 + n["d_xhat"] * m1) \
        + np.abs(refs[0]) * (n["rel"] + 2 * U)
    # a column's sum: rows of a workgroup one after the other, then the workgroups' sums
    dr = 64 + rows
    d_dw = dr * U * (np.abs(dy) * xh).sum(0) + (np.abs(dy) * n["d_xhat"]).sum(0)
    return refs, (d_dx, d_dw, dr * U * np.abs(dy).sum(0))


def lora_bounds(base, x, a, b, index, scales, dtype):
    """(y, h, error of y, error of h).  h's sum over K may be truncated (2 u a step); h enters the second product as
    two bf16 values (2^-17 of it) unless the type is binary32."""
    K, R = a.shape[2], a.shape[1]
    y, h = block.lora(base, x, a, b, index, scales)
    ah = block.lora(np.zeros_like(base), np.abs(x), np.abs(a), np.abs(b), index, np.abs(scales))[1]
    rep = 0.0 if dtype == torch.float32 else 2.0 ** -17
    d_h = (K + 24) * 2 * U * ah + rep * np.abs(h)
    wide = lambda t: through(t, np.abs(b), index, False)  # noqa: E731
    d_y = wide(d_h) + (2 * R + 24) * 2 * U * wide(np.abs(h)) + U * (np.abs(base) + np.abs(y))
    return y, h, d_y, d_h


def through(t, w, index, rows):
    """t (T, R) through |w| of each token's adapter: (T, C) with w (L, C, R), or (L, R, C) where rows."""
    out = np.zeros((t.shape[0], w.shape[2] if rows else w.shape[1]))
    for i in range(w.shape[0]):
        at = np.flatnonzero(index == i)
        out[at] = t[at] @ (w[i] if rows else w[i].T)
    return out


def lora_grad_bounds(dy, x, a, b, index, scales, h, d_h, dtype):
    """((dx, da, db), their errors)."""
    N, R = b.shape[1], a.shape[1]
    dx, da, db, g = block.lora_grads(dy, x, a, b, index, scales, h)
    ag = block.lora_grads(np.abs(dy), np.abs(x), np.abs(a), np.abs(b), index, np.abs(scales), np.abs(h))[3]
    # (an fp16 operand beside the two halves is two bf16 values too, without their smallest product)
    rep = 0.0 if dtype == torch.float32 else 2.0 ** -17
    d_g = (N + 24) * 2 * U * ag + rep * np.abs(g)
    d_dx = through(d_g, np.abs(a), index, True) + (2 * R + 24) * 2 * U * through(np.abs(g), np.abs(a), index, True)
    d_da, d_db = np.zeros_like(da), np.zeros_like(db)
    for i in range(a.shape[0]):
        at = np.flatnonzero(index == i)
        n = 3 * len(at) + 24
        d_da[i] = (d_g[at] + (n * 2 * U + rep) * np.abs(g[at])).T @ np.abs(x[at])
        d_db[i] = np.abs(dy[at]).T @ (d_h[at] + (n * 2 * U + rep) * np.abs(h[at]))
    return (dx, da, db), (d_dx, d_da, d_db)
