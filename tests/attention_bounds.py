"""Bounds of attention's rows against 64 bits, token by token, so that they hold
where keys or values of one sequence differ by any amount."""
import numpy as np

from oracle import attention as oa

UNIT = {"bfloat16": 2.0**-8, "float16": 2.0**-11}  # half a step, relative to the value


def near(y, q, batch, values, dtype, window=0, sinks=0, scale=None, rows=None):
    """Every row (of `rows`, a mask of tokens) against 64 bits.

    A score is off by the 32-bit sum over the head (dim + 8 additions of at most 2^-23 each of sum |q||k|, tensor cores
    truncate), by what the query's scaling into 16 bits loses (2^-24 of it) and by its factors (4 roundings of 2^-24): d
    in all.  A weight e^s is off by e^(d + the same of the largest) - 1, by 2^x and its sum (2 x 2^-21), by its rounding
    to 11 significant bits (half a step: 2^-11) for bfloat16 or to what two such leave (2^-22) for float16, by the 32-bit
    sums over the tokens (2^-23 for each 16 of them, and the joining) and, where it is below 2^-14 of the 16-bit range,
    by 2^-25 of that: the token that counts most has 2^-6 at least (lifted by 2^7; references are rounded up, 2, values'
    exponents follow late, 2^3, and a tile's are within 2^9), so by 2^-19 of what that one adds, times the size of its
    own element relative to its row.  (A row of zeros has no exponent: its weight counts as that of the largest row, as
    what comes next to it has 2^-25 of the range below its weight.)  Then the output's rounding."""
    y = y.double().cpu().numpy()
    qn = q.double().cpu().numpy()
    heads, group, dim = values[0].shape[1], q.shape[1] // values[0].shape[1], q.shape[2]
    scale = dim**-0.5 if scale is None else scale
    weight = 2.0**-11 if dtype == "bfloat16" else 2.0**-22
    for b, (length, _) in enumerate(batch.sizes):
        for i, p in enumerate(batch.positions(b)):
            t = batch.starts[b] + i
            if rows is not None and not rows[t]:
                continue
            j = np.flatnonzero(oa.sees(p, np.arange(max(length, 0)), window, sinks))
            if len(j) == 0:
                assert not y[t].any(), (b, i)
                continue
            for h in range(heads):
                k, v = values[b][:, h][:, j]
                x = qn[t, h * group : (h + 1) * group]
                s, d = x @ k.T * scale, (np.abs(x) @ np.abs(k).T) * abs(scale) * ((dim + 12) * 2.0**-23 + 2.0**-24)
                top = s.max(1, keepdims=True)
                d = np.minimum(d + np.take_along_axis(d, s.argmax(1)[:, None], 1), 700.0)
                with np.errstate(over="ignore"):
                    w, up = np.exp(s - top), np.exp(np.minimum(s - top + d, 700.0))
                z = w.sum(1, keepdims=True)
                w, off = w / z, (up - w) / z
                off = off + w * off.sum(1, keepdims=True) + w * (weight + 3 * 2.0**-21 + (length / 16 + 64) * 2.0**-23)
                size = np.abs(v)
                most = np.where(size.any(1), size.max(1), max(size.max(), 1e-300))
                want = w @ v
                err = off @ size + 2.0**-19 * (w * most).max(1, keepdims=True) * (size / most[:, None]).sum(0)
                bound = err * 1.01 + UNIT[dtype] * (np.abs(want) + err) + 2.0**-24 * (dtype == "float16") + 2.0**-133
                got = y[t, h * group : (h + 1) * group]
                assert np.isfinite(got).all(), (b, i, h)
                over = np.abs(got - want) - bound
                assert (over <= 0).all(), (b, i, h, np.unravel_index(over.argmax(), over.shape), over.max(), bound.max())
