"""Attention over the 4-bit cache where scores, keys and values are far from one:
large scores, rows and blocks of very different sizes."""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import attention as oa

from attention_bounds import UNIT, near
from attention_util import Batch, filled, queries

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp4", "nvfp4")
DTYPES = ("bfloat16", "float16")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,dim", (([(90, 1), (200, 1)], 64), ([(300, 3)], 256), ([(9001, 1)], 128), ([(90, 60), (600, 60)], 64), ([(300, 70)], 128), ([(4500, 80)], 64), ([(700, 50)], 256)))
def test_scores_of_any_size(fmt, dtype, sizes, dim):
    """Where one score is further above the others than they are off by, its token's value is the answer, whatever the
    scores' size: 2^x counts lifts and exponents of rows beside them."""
    batch = Batch(sizes, 16)
    cache, values = filled(batch, 1, dim, fmt, 2, lambda rng, shape: 2.0 ** rng.integers(-5, 6, shape))
    q = queries(batch, 2, dim, dtype)
    qn = q.double().cpu().numpy()
    for power in (5, 15, 20, 22, 24, 27, 30, 40, 60):
        for sign in (1.0, -1.0):
            y = ddg.mx4_attention(q, cache, *batch.dev, scale=sign * 2.0**power).double().cpu().numpy()
            alone = 0
            for b in range(len(sizes)):
                k, v = values[b][:, 0]
                for i, p in enumerate(batch.positions(b)):
                    s, size = sign * qn[batch.starts[b] + i] @ k[: p + 1].T, np.abs(qn[batch.starts[b] + i]) @ np.abs(k[: p + 1]).T
                    low, top = np.sort(s, 1)[:, -2:].T
                    # e^-30 of the others in all, and what both scores are off by (as in attention_bounds)
                    sure = (top - low) * 2.0**power > 30 + np.log(p + 1) + 2.0**power * 2 * size.max(1) * ((dim + 12) * 2.0**-23 + 2.0**-24)
                    want = v[s.argmax(1)]
                    got = y[batch.starts[b] + i]
                    assert np.isfinite(got).all(), (power, b, i)
                    off = np.abs(got - want) - (UNIT[dtype] + 2.0**-19) * np.abs(want) - 2.0**-12 * np.abs(v[: p + 1]).max() * np.exp(-30) - 2.0**-24 * (dtype == "float16")
                    assert (off[sure] <= 0).all(), (power, sign, b, i)
                    alone += sure.sum()
            assert alone > 0.8 * batch.tokens * 2 or power < 15, (power, alone)


def stored(batch, heads, dim, fmt, factors, seed=0):
    """(cache, values) of random rows times factors[b] (2, heads, length, dim or 1)."""
    it = iter(factors)
    return filled(batch, heads, dim, fmt, seed, lambda rng, shape: next(it))


SIZES = {"few": [(300, 1), (900, 3), (70, 10)], "many": [(300, 300), (900, 120), (70, 70)], "long": [(5000, 30)]}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,dim", (("few", 128), ("many", 64), ("many", 128), ("many", 256), ("long", 96)))
@pytest.mark.parametrize("far", (12, 45, 100))
def test_later_tokens_do_not_matter(fmt, dtype, sizes, dim, far):
    """Keys, values or both of some tokens 2^far times the others': the queries before them are what they are without."""
    batch = Batch(SIZES[sizes], 16)
    low = 1.0 if far < 100 else 2.0**-50
    factors, rows = [], []
    for b, (length, n) in enumerate(batch.sizes):
        f = np.full((2, 1, length, 1), low)
        for i, j in enumerate(range(length - n // 2 - 1, length, 29)):
            f[[0, 1] if i % 3 == 0 else i % 3 - 1, :, j] = low * 2.0**far
        factors.append(f)
        rows.append(batch.positions(b) < length - n // 2 - 1)
    cache, values = stored(batch, 2, dim, fmt, factors)
    q = queries(batch, 6, dim, dtype)
    y = ddg.mx4_attention(q, cache, *batch.dev, scale=dim**-0.5 / low)
    near(y, q, batch, values, dtype, scale=dim**-0.5 / low, rows=np.concatenate(rows))
    if dtype == "float16" and low < 1:
        assert not y[np.concatenate(rows)].any()  # 2^-50 in float16


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,dim", (("few", 128), ("many", 64), ("many", 128), ("many", 256), ("long", 96)))
def test_tokens_that_the_window_has_left_do_not_matter(fmt, sizes, dim):
    """Among the sinks' group, between sinks and window, just before it."""
    batch = Batch(SIZES[sizes], 16)
    window, sinks, factors = 64, 3, []
    for b, (length, n) in enumerate(batch.sizes):
        f = np.ones((2, 1, length, 1))
        first = length - n
        for j in (sinks, sinks + 1, 15, 16, first - window - 20, first - window):
            if sinks <= j <= first - window:
                f[:, :, j] = 2.0**70
        factors.append(f)
    cache, values = stored(batch, 2, dim, fmt, factors)
    q = queries(batch, 6, dim, "bfloat16")
    y = ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks)
    near(y, q, batch, values, "bfloat16", window, sinks)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,dim", (("few", 128), ("many", 64), ("many", 128), ("many", 256), ("long", 96)))
@pytest.mark.parametrize("spread", (3, 10, 30, 60))
def test_rows_of_any_size(fmt, dtype, sizes, dim, spread):
    """Values over 2^+-spread, the larger ones with the smaller weights; keys of 2^-2 spread and more; rows of zeros."""
    batch = Batch(SIZES[sizes], 16)
    rng = np.random.default_rng(spread)
    factors = []
    for length, _ in batch.sizes:
        f = np.stack((2.0 ** rng.integers(-2 * spread, 1, (2, length, 1)), 2.0 ** rng.integers(-spread, spread + 1, (2, length, 1))))
        f[0, :, rng.integers(0, length, 9)] = 0
        f[1, :, rng.integers(0, length, 9)] = 0
        f[:, :, 128:256] *= rng.integers(0, 2)  # a tile of zeros or none
        if dtype == "float16":
            f[1] = np.minimum(f[1], 2.0**10)
        factors.append(f)
    cache, values = stored(batch, 2, dim, fmt, factors)
    # keys that point away from every query where values are large: weights of about 2^-(their exponent) and less
    q = queries(batch, 6, dim, dtype)
    y = ddg.mx4_attention(q, cache, *batch.dev)
    near(y, q, batch, values, dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", (1, 40, 300))
def test_large_values_of_small_weight(fmt, n):
    """A token of weight 2^-60 whose value is 2^60 or 2^64 times the others' counts as much as they do, or most."""
    batch, dim = Batch([(300, n), (700, 2)], 16), 64
    import torch
    for power in (56, 60, 64):
        cache = ddg.mx4_cache(batch.pages, 16, 1, dim, fmt)
        values, x = [], np.zeros((batch.tokens, 1, dim))
        k, v = [np.zeros((n_, 1, dim)) for n_, _ in batch.sizes], [np.zeros((n_, 1, dim)) for n_, _ in batch.sizes]
        rng = np.random.default_rng(1)
        for b, (length, _) in enumerate(batch.sizes):
            v[b][:] = rng.choice((1.0, 1.5, 2.0, -3.0), v[b].shape)
            k[b][:, 0, 0] = 0.0
            for j in (0, 7, 130, 290):
                if j < length:
                    k[b][j, 0, 0] = -6.0  # scores 10 below the others' in the exponent of e, 6 times
                    v[b][j] *= 2.0**power
        starts = np.cumsum([0] + [len(a) for a in k]).astype(np.int32)
        every = [torch.from_numpy(starts).cuda(), batch.dev[1], batch.dev[2]]
        flat = [torch.from_numpy(np.concatenate(t)).float().cuda() for t in (k, v)]
        ddg.mx4_cache_append(cache, *flat, *every)
        kk, vv = (t.double().cpu().numpy() for t in ddg.mx4_cache_read(cache, int(starts[-1]), *every, dtype=torch.float32))
        values = [np.stack((kk[a:e], vv[a:e])).transpose(0, 2, 1, 3) for a, e in zip(starts, starts[1:])]
        x[..., 0] = 1.0
        q = torch.from_numpy(x).bfloat16().cuda()
        scale = 60 * np.log(2.0) / 6.0
        y = ddg.mx4_attention(q, cache, *batch.dev, scale=scale)
        near(y, q, batch, values, "bfloat16", scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,dim", (("few", 128), ("many", 64), ("many", 128), ("many", 256), ("long", 200)))
def test_blocks_of_very_different_sizes(fmt, dtype, sizes, dim):
    """Blocks of a row down to 2^-27 of its largest (nvfp4 has 2^-17): each channel to its own size, and keys whose
    query looks at the small blocks only."""
    batch = Batch(SIZES[sizes], 16)
    block = 32 if fmt == "mxfp4" else 16
    least = -27 if fmt == "mxfp4" else -12
    rng = np.random.default_rng(3)
    powers = np.linspace(0, least, -(-dim // block)).round()
    factors = []
    for length, _ in batch.sizes:
        f = 2.0 ** np.broadcast_to(np.repeat(powers, block)[:dim], (2, 2, length, dim)) * 2.0 ** rng.integers(-4, 1, (2, 2, length, 1))
        factors.append(f * (2.0**8 if dtype == "float16" else 1.0))
    cache, values = stored(batch, 2, dim, fmt, factors)
    q = queries(batch, 4, dim, dtype)
    y = ddg.mx4_attention(q, cache, *batch.dev)
    near(y, q, batch, values, dtype)
    if dtype == "bfloat16":  # a query of the least block alone, as large as the keys there are small
        q[..., : (len(powers) - 1) * block] = 0
        q *= 2.0**-least
        near(ddg.mx4_attention(q, cache, *batch.dev), q, batch, values, dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", (64, 96, 256))
def test_what_else_such_items_have(fmt, dim):
    """Items with rows far apart: NaN in values of a token and a page that is not there reach the queries that see them
    alone, rows of no sequence stay, unaligned and strided operands, equal bits call for call and in a captured graph."""
    import torch
    batch = Batch([(300, 200), (1100, 90), (90, 60)], 16, lead=2, tail=3)
    factors = []
    for length, _ in batch.sizes:
        f = np.ones((2, 1, length, 1))
        f[:, :, length - 7] = 2.0**40
        f[:, :, length // 2 :: 31] *= 2.0**-20
        factors.append(f)
    cache, values = stored(batch, 2, dim, fmt, factors)
    q = queries(batch, 8, dim, "bfloat16")
    p = np.concatenate([np.full(batch.starts[0], -1)] + [batch.positions(b) for b in range(3)] + [np.full(3, -1)])
    b_of = np.concatenate([np.full(batch.starts[0], -1)] + [np.full(n, b) for b, (_, n) in enumerate(batch.sizes)] + [np.full(3, -1)])
    before = np.concatenate([[False] * batch.starts[0]] + [batch.positions(b) < length - 7 for b, (length, _) in enumerate(batch.sizes)] + [[False] * 3])
    want = torch.full_like(q, 5.0)
    ddg.mx4_attention(q, cache, *batch.dev, out=want)
    near(want, q, batch, values, "bfloat16", rows=before)
    assert (want[: batch.starts[0]] == 5).all() and (want[-3:] == 5).all()
    # strides, and one element off 16 bytes
    odd = torch.zeros(batch.tokens * 8 * (dim + 1) + 1, dtype=torch.bfloat16, device="cuda")[1:].view(batch.tokens, 8, dim + 1)
    odd[..., :dim] = q
    out = torch.full((8, batch.tokens, dim), 5.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(ddg.mx4_attention(odd[..., :dim], cache, *batch.dev, out=out), want)
    ddg.mx4_attention(q, cache, *batch.dev, out=odd[..., :dim])
    mine = slice(batch.starts[0], batch.starts[-1])
    assert torch.equal(odd[mine, :, :dim], want[mine]) and not odd[..., dim].any()
    graph, again = torch.cuda.CUDAGraph(), torch.full_like(q, 5.0)
    with torch.cuda.graph(graph):
        ddg.mx4_attention(q, cache, *batch.dev, out=again)
    for _ in range(3):
        again.fill_(5.0)
        graph.replay()
        assert torch.equal(again, want)
    # NaN in a block of a token's values
    size = 32 if fmt == "mxfp4" else 16
    page, off = batch.place(0, 150)
    cache.scales[page, 1, 1, off, 1] = 255 if fmt == "mxfp4" else 127
    y = ddg.mx4_attention(q, cache, *batch.dev)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[torch.from_numpy((b_of == 0) & (p >= 150)).cuda(), 4:, size : 2 * size] = True
    assert torch.equal(torch.isnan(y[mine]), bad[mine]) and torch.equal(torch.where(bad, 0.0, y)[mine], torch.where(bad, 0.0, want)[mine])
    # a page that is not there
    table = batch.dev[2].clone()
    table[1, 64] = -1  # tokens 1024 to 1039
    y = ddg.mx4_attention(q, cache, *batch.dev[:2], table)
    lost = torch.from_numpy((b_of == 1) & (p >= 1024)).cuda()
    assert torch.isnan(y[lost]).all()
    kept = torch.from_numpy(b_of >= 0).cuda() & ~lost
    assert torch.equal(torch.isnan(y[kept]), bad[kept])


def test_no_wait_gave_up_in_these():
    assert ddg.wait_timeouts() == 0
