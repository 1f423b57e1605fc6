"""Rotary positions, the paged 4-bit cache and attention over it, in 64 bits
(numpy), written from their definitions in include/ddgemm.h and independent of the
library.
"""
import numpy as np

from . import microscaled as ms


def angles(positions, turns):
    """2 pi frac(p t / 2^64), with the fraction exact: (tokens, pairs)."""
    f = np.array([[(int(p) * int(t)) % (1 << 64) for t in turns] for p in positions], dtype=object).reshape(len(positions), len(turns))
    return np.array(f / (1 << 64), dtype=np.float64) * (2 * np.pi)


def rotary(x, positions, turns, scale=1.0, interleaved=False, inverse=False):
    """x (tokens, heads, dim)."""
    x = np.asarray(x, dtype=np.float64)
    n = len(turns)
    a = angles(positions, turns)[:, None]
    c, s = scale * np.cos(a), scale * np.sin(a) * (-1 if inverse else 1)
    y = x.copy()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def width_of(dim):
    return 64 if dim <= 64 else 128 if dim <= 128 else 256


def rows(x, fmt):
    """Rows x (n, dim) as the cache stores them: (codes (n, width / 2), scales
    (n, width / block), exponents (n))."""
    x = np.asarray(x, dtype=np.float64)
    n, dim = x.shape
    code, byte, exps = ms.quantize(np.pad(x, ((0, 0), (0, width_of(dim) - dim))), fmt)
    code = code.reshape(n, -1)
    if fmt == "mxfp4":
        exps = np.where(byte == 255, 0, byte).max(axis=1).astype(np.int32) - 127
    else:
        exps = np.where(np.where(np.isfinite(x), x, 0).any(axis=1), exps, -127)
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8), byte, exps.astype(np.int8)


def row_values(codes, scales, exponents, fmt, dim):
    """The values of stored rows, (n, dim)."""
    code = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1, ms.BLOCK[fmt]).astype(np.int64)
    return ms.values(code, scales, exponents.astype(np.int64), fmt, code.shape[1] * code.shape[2])[:, :dim]


def sees(p, j, window=0, sinks=0):
    return (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))


def attention(q, k, v, positions, scale, window=0, sinks=0):
    """One head: q (n, dim) at `positions`, k and v (length, dim) of one sequence.
    (outputs (n, dim), the same with |v|, the largest |score|'s bound sum |q||k| scale
    over the tokens seen); a row that sees nothing is 0."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    j = np.arange(k.shape[0])
    y, size, most = np.zeros_like(q), np.zeros_like(q), np.zeros(len(q))
    for i, p in enumerate(positions):
        at = np.flatnonzero(sees(p, j, window, sinks))
        if len(at) == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            s = k[at] @ q[i] * scale
            w = np.exp(s - s.max())
            w = w / w.sum()
            y[i], size[i] = w @ v[at], w @ np.abs(v[at])
            most[i] = (np.abs(k[at]) @ np.abs(q[i])).max() * abs(scale)
    return y, size, most
