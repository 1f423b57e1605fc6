"""The 4-bit microscaled formats, element by element in exact arithmetic
(numpy float64: every comparison below is between numbers of few significant
bits and is exact), and the gated feed-forward block in 64 bits.

Independent of the library: formats, layouts and roundings are written from
their definition in include/ddgemm.h.
"""
import math

import numpy as np

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def e4m3_grid():
    """The finite E4M3 magnitudes by byte, 0 .. 126 (127 is NaN)."""
    return np.array([(b % 8) * 2.0**-9 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 10) for b in range(127)])


def nearest_code(ratio_num, unit):
    """Index of the code nearest to ratio_num / unit >= 0, ties to the even
    index, saturating: comparisons of ratio_num with midpoint * unit."""
    code = np.zeros(ratio_num.shape, dtype=np.int64)
    for i in range(7):
        edge = (CODES[i] + CODES[i + 1]) / 2 * unit
        code += (ratio_num >= edge) if i % 2 else (ratio_num > edge)
    return code


def quantize(x, fmt):
    """(codes 0..15 (rows, blocks, size), scale bytes (rows, blocks), row exponents)
    of x (rows, k); the last block is filled up with zeros."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    size = BLOCK[fmt]
    x = np.pad(x, ((0, 0), (0, -k % size))).reshape(rows, -1, size)
    most = np.abs(x).max(axis=2, initial=0.0)
    broken = ~np.isfinite(x).all(axis=2)
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    with np.errstate(invalid="ignore", over="ignore"):
        if fmt == "mxfp4":
            _, e = np.frexp(np.where(broken, 1.0, most))
            byte = np.where(most > 0, np.clip(e - 1 - 2 + 127, 0, 255), 0)
            unit = np.ldexp(1.0, byte - 127)
            byte = np.where(broken, 255, byte)
            exps = np.zeros(rows, dtype=np.int32)
        else:
            top = finite.reshape(rows, -1).max(axis=1, initial=0.0)
            exps = np.zeros(rows, dtype=np.int32)
            for r in range(rows):
                if top[r] > 0:
                    e = math.frexp(top[r])[1] - 14
                    while top[r] > 2688 * 2.0**e:
                        e += 1
                    exps[r] = max(e, -100)
            grid = e4m3_grid()
            amax = np.where(broken, 0.0, most)
            six = 6.0 * np.ldexp(1.0, exps)[:, None]
            byte = np.zeros(amax.shape, dtype=np.int64)
            for b in range(126):  # ties between b and b + 1 go to the even byte
                edge = (grid[b] + grid[b + 1]) / 2 * six
                byte += (amax >= edge) if b % 2 else (amax > edge)
            byte = np.where((amax > 0) & (byte == 0), 1, byte)
            unit = grid[byte] * np.ldexp(1.0, exps)[:, None]
            byte = np.where(broken, 127, byte)
        code = nearest_code(np.where(np.isfinite(x), np.abs(x), 0.0), np.where(unit > 0, unit, 1.0)[..., None])
    code = code | (np.signbit(x).astype(np.int64) << 3)
    return code, byte.astype(np.uint8), exps


def values(code, byte, exps, fmt, k):
    """The values of quantize()'s result, (rows, k); NaN in blocks whose scale is."""
    v = CODES[code & 7] * np.where(code >> 3, -1.0, 1.0)
    if fmt == "mxfp4":
        scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    else:
        scale = np.append(e4m3_grid(), np.nan)[byte] * np.ldexp(1.0, exps)[:, None]
    return (v * scale[..., None]).reshape(v.shape[0], -1)[:, :k]


def scale_offset(row, block, fmt, k):
    """Byte offset of a scale in the tiled layout."""
    per_row = -(-k // 256) * (256 // BLOCK[fmt] // 4)
    return (row // 128 * per_row + block // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + block % 4


def activation(g, act):
    """act(g) and act'(g) in float64."""
    erf = np.vectorize(math.erf, otypes=[np.float64])
    if act == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = 0.5 * (1 + erf(g / math.sqrt(2)))
        return g * c, c + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = np.tanh(k * (g + 0.044715 * g**3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    return np.maximum(g, 0.0), (g > 0).astype(np.float64)


def gated(x, wg, wu, wd, act, dy=None):
    """y of the gated block, or with dy a dict of y, its intermediates and gradients."""
    x, wg, wu, wd = (np.asarray(t, dtype=np.float64) for t in (x, wg, wu, wd))
    g, u = x @ wg.T, x @ wu.T
    a, da = activation(g, act)
    h = a * u
    y = h @ wd.T
    if dy is None:
        return y
    dy = np.asarray(dy, dtype=np.float64)
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return {"y": y, "g": g, "u": u, "a": a, "da": da, "h": h, "dh": dh, "dg": dg, "du": du,
            "dx": dg @ wg + du @ wu, "dwg": dg.T @ x, "dwu": du.T @ x, "dwd": dy.T @ h}
