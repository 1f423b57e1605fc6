"""What rows that no query sees hold does not matter to attention, whatever their
bytes: rows behind a sequence's end, of pages that no sequence has, of later tokens."""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg

from attention_bounds import near
from attention_util import Batch, filled, queries

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp4", "nvfp4")
DTYPES = ("bfloat16", "float16")


def no_token(batch):
    """Which rows (pages, page_size) of the cache no sequence has."""
    free = np.ones((batch.pages, batch.page), dtype=bool)
    for b, (length, _) in enumerate(batch.sizes):
        for j in range(length):
            free[batch.place(b, j)] = False
    return free


def bytes_of(kind, rng, shape):
    if kind == "any":
        return rng.integers(0, 256, shape)
    return np.full(shape, kind)


# (codes, scales, exponents) of the rows: memory that was not cleared, scales that do not belong to their exponent
FILLS = ((0, 0, 0), (0xCD, 0xCD, 0xCD), ("any", 254, 0), ("any", 0x7E, 0x7F), ("any", "any", 0x81), ("any", "any", 0x80), ("any", "any", "any"), (0xFF, 0xFF, 0xFF))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", (64, 100, 128, 256))
@pytest.mark.parametrize("n", (1, 3, 60))
def test_rows_that_no_token_has(fmt, dtype, dim, n):
    import torch
    batch = Batch([(200, n), (77, n), (2500, 1), (65, n), (n, n)], 64, seed=dim)
    cache, values = filled(batch, 2, dim, fmt, dim)
    q = queries(batch, 8, dim, dtype)
    free = torch.from_numpy(no_token(batch)).cuda()
    rng = np.random.default_rng(n)
    parts = (cache.codes, cache.scales, cache.exponents)
    for window, sinks in ((0, 0), (50, 3)):
        want = None
        for kinds in FILLS:
            for t, kind in zip(parts, kinds):
                bytes_ = torch.from_numpy(bytes_of(kind, rng, tuple(t.shape)).astype(np.uint8)).cuda().view(t.dtype)
                t.copy_(torch.where(free[:, None, None].reshape(free.shape[0], 1, 1, free.shape[1], *[1] * (t.dim() - 4)), bytes_, t))
            y = ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks)
            if want is None:
                near(y, q, batch, values, dtype, window, sinks)
                want = y
            assert torch.equal(y, want), (kinds, window)
    assert ddg.wait_timeouts() == 0


@pytest.mark.parametrize("group", (1, 4))
@pytest.mark.parametrize("window,sinks", ((1, 0), (1, 4), (7, 3), (16, 4), (16, 40), (100, 0), (100, 4), (300, 20), (5000, 1)))
@pytest.mark.parametrize("n", (1, 11, 40, 300))
def test_page_tables_that_end_before_the_window(n, window, sinks, group):
    """A query beyond the table does not see itself: NaN, sinks or none.  Those within it are what they are without."""
    import torch
    batch = Batch([(400, n), (3000, 1), (40, 1)], 16, table_pad=0)
    cache, values = filled(batch, 1, 64, "mxfp4")
    q = queries(batch, group, 64, "bfloat16")
    want = ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks)
    near(want, q, batch, values, "bfloat16", window, sinks)
    p = np.concatenate([batch.positions(b) for b in range(3)])
    for pages in (1, 2, 4, 9, 18, 24):
        y = ddg.mx4_attention(q, cache, *batch.dev[:2], batch.dev[2][:, :pages].contiguous(), window=window, sinks=sinks)
        hit = torch.from_numpy(p >= 16 * pages)
        assert torch.isnan(y[hit]).all(), pages
        near(y, q, batch, values, "bfloat16", window, sinks, rows=~hit.numpy())  # parts may be others
    far = batch.dev[1].clone()
    for length in (10000, (1 << 31) - 1):
        far[0] = length
        y = ddg.mx4_attention(q, cache, batch.dev[0], far, batch.dev[2], window=window, sinks=sinks)
        assert torch.isnan(y[:n]).all() and torch.equal(y[n:], want[n:]), length  # the same table, the same parts


@pytest.mark.parametrize("n", (1, 5, 60, 700))
@pytest.mark.parametrize("length", (-1, -5, -(1 << 28), -(1 << 31) + 3, -(1 << 31)))
def test_lengths_far_below_zero(n, length):
    """Every position is negative: nothing is written, read as NaN, and queries see nothing (lengths - n would overflow)."""
    import torch
    batch = Batch([(max(n, 40), n), (90, 2)], 16)
    cache, values = filled(batch, 2, 64, "nvfp4")
    before = [t.clone() for t in (cache.codes, cache.scales, cache.exponents)]
    lengths = batch.dev[1].clone()
    lengths[0] = length
    plan = (batch.dev[0], lengths, batch.dev[2])
    k, v = (torch.randn(batch.tokens, 2, 64, device="cuda").bfloat16() for _ in range(2))
    got = torch.stack(ddg.mx4_cache_read(cache, batch.tokens, *plan))
    assert torch.isnan(got[:, :n]).all() and torch.isfinite(got[:, n:]).all()
    for window, sinks in ((0, 0), (20, 3)):
        y = ddg.mx4_attention(queries(batch, 8, 64, "bfloat16"), cache, *plan, window=window, sinks=sinks)
        assert not y[:n].any() and torch.isfinite(y[n:]).all() and y[n:].any()
    starts = torch.tensor([0, n, n], dtype=torch.int32, device="cuda")  # of the first sequence alone
    ddg.mx4_cache_append(cache, k[:n], v[:n], starts, lengths, batch.dev[2], rotary=ddg.rotary_table(64))
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.codes, cache.scales, cache.exponents)))
