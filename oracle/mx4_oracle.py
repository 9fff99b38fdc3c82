"""Oracle of the microscaled 4-bit form and of the mixture-of-experts layer
(numpy, binary64; OCP Microscaling Formats 1.0, MXFP4).

Blocks of 32 along K: E = clamp(floor(log2 max|x|) - 2, -127, 125), codes x / 2^E
to the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} (ties to the even code, saturating),
scale byte E + 127; zeros give byte 0, a non-finite value byte 255.
"""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def code_bytes(rows, K):
    return rows * 16 * ((K + 31) // 32)


def scale_bytes(rows, K):
    return 512 * ((rows + 127) // 128) * ((K + 127) // 128)


def quantise(x):
    """x [rows, K] (any float type) -> codes uint8 [rows, Kp], bytes uint8 [rows, Kp / 32]."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    kp = (K + 31) // 32 * 32
    b = np.zeros((rows, kp))
    b[:, :K] = x
    b = b.reshape(rows, kp // 32, 32)
    bad = ~np.isfinite(b).all(2)
    safe = np.where(bad[:, :, None], 0.0, b)
    a = np.abs(safe).max(2)
    E = np.where(a > 0, np.frexp(a)[1] - 3, -127).clip(-127, 125)
    v = np.ldexp(np.abs(safe), -E[:, :, None])
    mids = (GRID[1:] + GRID[:-1]) / 2
    # number of midpoints below v; a midpoint itself goes to the even code
    c = (v[..., None] > mids).sum(-1)
    tie = (v[..., None] == mids).any(-1)
    c = np.where(tie & (c % 2 == 1), c + 1, c)
    c = c + 8 * np.signbit(safe)
    c = np.where(bad[:, :, None], 0, c)
    byte = np.where(bad, 255, E + 127)
    return c.reshape(rows, kp).astype(np.uint8), byte.astype(np.uint8)


def pack(codes, byte):
    """-> packed uint8 [rows, Kp / 2], tiled scales uint8 [scale_bytes]."""
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    rows, kb = byte.shape
    kqs = (kb + 3) // 4
    t = np.zeros(scale_bytes(rows, kb * 32), np.uint8)
    for r in range(rows):
        for b in range(kb):
            t[((r // 128) * kqs + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte[r, b]
    return packed, t


def values(codes, byte, K):
    """binary64 [rows, K]."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    rows = v.shape[0]
    E = byte.astype(np.int64) - 127
    v = np.ldexp(v.reshape(rows, -1, 32), E[:, :, None])
    v = np.where((byte == 255)[:, :, None], np.nan, v)
    return v.reshape(rows, -1)[:, :K]


def roundtrip(x):
    c, b = quantise(x)
    return values(c, b, np.shape(x)[1])


def route(x, router, topk, renorm):
    """-> experts int [T, topk], probs binary64 [T, topk]; NaN logits last, ties to the lowest."""
    with np.errstate(invalid="ignore", over="ignore"):
        logits = np.einsum("th,eh->te", x.astype(np.float64), router.astype(np.float64))
    T, E = logits.shape
    key = np.where(np.isnan(logits), -np.inf, logits)
    ids = np.zeros((T, topk), np.int64)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (bool(np.isnan(logits[t, e])), -key[t, e], e))
        ids[t] = order[:topk]
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.take_along_axis(logits, ids, 1)
        num = np.exp(top - top[:, :1])
        den = num.sum(1, keepdims=True) if renorm else np.exp(logits - top[:, :1]).sum(1, keepdims=True)
        return ids, num / den


def moe(x, router, w13, w2, topk, renorm):
    """x [T, H], w13 [E, 2 I, H] (gate and up rows interleaved), w2 [E, H, I], all
    binary64 values -> (Y, experts, probs, A), A the sum over i of p |down| |h|."""
    ids, p = route(x, router, topk, renorm)
    T = x.shape[0]
    y = np.zeros((T, w2.shape[1]))
    A = np.zeros_like(y)
    for t in range(T):
        for j in range(topk):
            e = ids[t, j]
            gu = w13[e] @ x[t]
            g, u = gu[0::2], gu[1::2]
            with np.errstate(over="ignore"):
                h = g / (1 + np.exp(-g)) * u
            y[t] += p[t, j] * (w2[e] @ h)
            A[t] += p[t, j] * (np.abs(w2[e]) @ np.abs(h))
    return y, ids, p, A
