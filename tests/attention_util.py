"""Batches, caches and bounds for the tests of attention over the 4-bit cache."""
import numpy as np

import extended_precision_gemm_gb300 as ddg
from oracle import attention as oa

UNIT = {"bfloat16": 2.0**-8, "float16": 2.0**-11, "float32": 2.0**-24}


class Batch:
    """Sequences of (length, new tokens) whose pages lie in any order in a cache of
    `spare` pages more than they need; `lead` and `tail` tokens of no sequence."""

    def __init__(self, sizes, page, seed=0, lead=0, tail=0, spare=2, table_pad=1):
        import torch
        rng = np.random.default_rng(seed)
        self.sizes, self.page = sizes, page
        need = [-(-max(n, 0) // page) for n, _ in sizes]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(sizes), max(need + [0]) + table_pad), -1, dtype=np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = order[sum(need[:b]):][:n]
        self.starts = np.cumsum([lead] + [n for _, n in sizes]).astype(np.int32)
        self.lengths = np.array([n for n, _ in sizes], dtype=np.int32)
        self.tokens = int(self.starts[-1]) + tail
        self.dev = [torch.from_numpy(x).cuda() for x in (self.starts, self.lengths, self.table)]

    def positions(self, b):
        n = self.starts[b + 1] - self.starts[b]
        return np.arange(self.lengths[b] - n, self.lengths[b])

    def place(self, b, j):
        """(page, offset) of token j of sequence b."""
        return self.table[b, j // self.page], j % self.page


def filled(batch, heads, dim, fmt, seed=0, sizes=None):
    """(cache, keys and values by sequence (2, heads, length, dim) in 64 bits): random
    rows, `sizes(rng, shape)` factors of them; rows that no sequence has hold NaN."""
    import torch
    rng = np.random.default_rng(seed + 1)
    cache = ddg.mx4_cache(batch.pages, batch.page, heads, dim, fmt)
    parts = [cache.codes.cpu().numpy(), cache.scales.cpu().numpy(), cache.exponents.cpu().numpy()]
    parts[0][:] = rng.integers(0, 256, parts[0].shape)
    parts[1][:] = 255 if fmt == "mxfp4" else 127
    values = []
    for b, (length, _) in enumerate(batch.sizes):
        x = rng.standard_normal((2, heads, max(length, 0), dim)) * np.exp(0.5 * rng.standard_normal((2, heads, 1, dim)))
        if sizes is not None:
            x = x * sizes(rng, (2, heads, max(length, 0), 1))
        if length <= 0:
            values.append(x)
            continue
        stored = oa.rows(x.astype(np.float32).reshape(-1, dim), fmt)
        back = oa.row_values(*stored, fmt, dim).reshape(x.shape)
        for j in range(length):
            page, off = batch.place(b, j)
            for part, rows in zip(parts, stored):
                part[page, :, :, off] = rows.reshape(*x.shape[:3], *rows.shape[1:])[:, :, j]
        values.append(back)
    cache.codes, cache.scales, cache.exponents = (torch.from_numpy(p).cuda() for p in parts)
    return cache, values


def queries(batch, heads, dim, dtype, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn(batch.tokens, heads, dim, generator=g).to(getattr(torch, dtype)).cuda()


def check(y, q, batch, values, dtype, window=0, sinks=0, scale=None, skip=()):
    """Every row against 64 bits.  The bound: a score is off by the 32-bit sum over the
    head (dim + 8 additions of at most 2^-23 each, tensor cores truncate, of sum |q||k|),
    what the scaling into 16 bits loses (2^-24 of it), and its factors (4 roundings),
    in the exponent of a weight; a weight by that, by 2^x (2^-21 and 2^-21 for the sum's), by
    its rounding to 16 bits (half a step of 11 bits, or 22 for float16) and by the 32-bit sums over the
    tokens (2^-23 for each 16 of them in a row of at most length / 16, and the joining); then the
    output's rounding."""
    y = y.double().cpu().numpy()
    heads = values[0].shape[1]
    group = q.shape[1] // heads
    dim = q.shape[2]
    scale = dim**-0.5 if scale is None else scale
    qn = q.double().cpu().numpy()
    for b, (length, n) in enumerate(batch.sizes):
        rows = slice(batch.starts[b], batch.starts[b + 1])
        for h in range(q.shape[1]):
            if (b, h) in skip:
                continue
            k, v = values[b][:, h // group]
            want, size, most = oa.attention(qn[rows, h], k, v, batch.positions(b), scale, window, sinks)
            weight = 2.0**-12 if dtype == "bfloat16" else 2.0**-22
            err = (2 * ((dim + 12) * 2.0**-23 + 2.0**-24) * most + weight + 3 * 2.0**-21 + (length / 16 + 64) * 2.0**-23)[:, None] * size
            bound = err * 1.01 + UNIT[dtype] * (np.abs(want) + err) + length * 2.0**-31 * size.max(initial=0.0) + 2.0**-24 * (dtype == "float16") + 2.0**-133
            got = y[rows, h]
            assert np.isfinite(got).all(), (b, h)
            off = np.abs(got - want) - bound
            assert (off <= 0).all(), (b, h, np.unravel_index(off.argmax(), off.shape), off.max(), bound.max())
