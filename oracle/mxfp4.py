"""Plain MXFP4 and gradient-norm arithmetic in binary64 (numpy), straight from the definitions.

Shares no code with the GPU path.  Inputs are arrays of values that binary64 holds exactly (bf16, fp16, fp32); every
step below -- frexp, division by a power of two, comparison with the midpoints of the e2m1 grid -- is exact.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MID = (GRID[1:] + GRID[:-1]) / 2  # a magnitude above MID[i] is nearer GRID[i + 1]; one on it goes to the even code
NAN = 255


def quantize(x, rule="floor"):
    """x (rows, cols) -> codes (rows, nb * 32) in 0..15 (zero past cols) and scales (rows, nb) in 0..255."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    m = np.abs(b).max(axis=2) if b.size else np.zeros((rows, nb))
    bad = ~np.isfinite(m)
    mant, expo = np.frexp(np.where(bad | (m == 0), 1.0, m))  # m = mant * 2^expo, 0.5 <= mant < 1
    e = expo - 1 - 2 + 127
    if rule == "ceil":
        e = e + (mant > 0.75)  # m > 1.5 * 2^(expo - 1): above 6 * 2^(expo - 3)
    e = np.where(m == 0, 0, np.maximum(e, 0))
    a = np.abs(np.where(bad[:, :, None], 0.0, b)) / np.exp2(e - 127.0)[:, :, None]
    code = np.zeros(a.shape, dtype=np.int64)
    for i, mid in enumerate(MID):
        code += (a >= mid) if i % 2 else (a > mid)  # code i + 1 is even when i is odd: a tie goes up to it
    code = np.where(np.signbit(b) & ~bad[:, :, None], code + 8, code)
    return code.reshape(rows, nb * 32).astype(np.uint8), np.where(bad, NAN, e).astype(np.uint8)


def values(codes, scales, cols):
    """The (rows, cols) values that codes (rows, nb * 32) and scales (rows, nb) stand for."""
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = np.where(scales == NAN, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v * np.repeat(s, 32, axis=1))[:, :cols]


def rounded(x, rule="floor"):
    x = np.asarray(x, dtype=np.float64)
    return values(*quantize(x, rule), x.shape[1])


def unpack(codes):
    """Packed bytes (rows, n) -> codes (rows, 2 n)."""
    return np.stack([codes & 15, codes >> 4], axis=2).reshape(codes.shape[0], -1)


def pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def norm(arrays, p):
    """Norm of all elements of a list of arrays as one vector."""
    parts = [np.abs(np.asarray(a, dtype=np.float64)).ravel() for a in arrays]
    flat = np.concatenate(parts) if parts else np.zeros(0)
    if flat.size == 0:
        return 0.0
    if p == 2.0:
        return float(np.sqrt(np.sum(flat * flat)))
    return float(flat.sum()) if p == 1.0 else float(flat.max())
