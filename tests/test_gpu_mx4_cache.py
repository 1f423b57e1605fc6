"""The paged 4-bit cache: rows written bit for bit as the oracle's, and read back."""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import attention as oa

from attention_util import Batch

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp4", "nvfp4")


def marked(batch, heads, dim, fmt):
    """A cache of bytes that no test writes by chance everywhere."""
    cache = ddg.mx4_cache(batch.pages, batch.page, heads, dim, fmt)
    cache.codes.fill_(0xA5)
    cache.scales.fill_(0x3C)
    cache.exponents.fill_(0x5A)
    return cache


def expect(cache, batch, k, v, fmt):
    """The three arrays after the append of k and v (tokens, heads, dim in 64 bits) to a marked cache."""
    parts = [np.full(tuple(t.shape), m, dtype=np.uint8) for t, m in ((cache.codes, 0xA5), (cache.scales, 0x3C), (cache.exponents, 0x5A))]
    for b in range(len(batch.sizes)):
        for i, p in enumerate(batch.positions(b)):
            if p < 0 or p // batch.page >= batch.table.shape[1] or not 0 <= batch.table[b, p // batch.page] < batch.pages:
                continue
            page, off = batch.place(b, p)
            for kv, x in enumerate((k, v)):
                for part, rows in zip(parts, oa.rows(x[batch.starts[b] + i], fmt)):
                    part[page, kv, :, off] = rows.view(np.uint8) if rows.dtype == np.int8 else rows
    return parts


def same(cache, parts):
    for t, want in zip((cache.codes, cache.scales, cache.exponents), parts):
        got = t.cpu().numpy().view(np.uint8)
        assert np.array_equal(got, want), np.argwhere(got != want)[:5]


def unsigned_zeros(codes):
    """Bytes of two codes with -0 (8) as 0: the same number, which of the two a zero becomes is not defined."""
    low, high = codes & 15, codes >> 4
    return np.where(low == 8, 0, low) | np.where(high == 8, 0, high) << 4


SIZES = [(40, 3), (1, 1), (17, 17), (5, 0), (0, 0), (33, 1)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ("float32", "bfloat16", "float16"))
@pytest.mark.parametrize("heads,dim,page", ((1, 64, 16), (3, 128, 16), (2, 256, 32), (5, 96, 64), (2, 80, 16), (1, 1, 16), (3, 40, 128), (2, 200, 16)))
def test_rows_are_the_oracles(fmt, dtype, heads, dim, page):
    import torch
    batch = Batch(SIZES, page, seed=dim, lead=2, tail=3)
    g = torch.Generator().manual_seed(dim)
    k, v = ((torch.randn(batch.tokens, heads, dim, generator=g) * torch.exp(2 * torch.randn(batch.tokens, heads, 1, generator=g))).to(getattr(torch, dtype)) for _ in range(2))
    k[3], v[4, 0] = 0, 0
    cache = marked(batch, heads, dim, fmt)
    assert ddg.mx4_cache_append(cache, k.cuda(), v.cuda(), *batch.dev) is cache
    want = expect(cache, batch, k.double().numpy(), v.double().numpy(), fmt)
    same(cache, want)
    # and back, exactly, in every type; rows of no sequence stay
    for back in (torch.float32, torch.bfloat16):
        out = tuple(torch.full((batch.tokens, heads, dim), 7.0, dtype=back).cuda() for _ in range(2))
        got = ddg.mx4_cache_read(cache, batch.tokens, *batch.dev, out=out)
        assert got[0] is out[0] and got[1] is out[1]
        for x, y in zip((k, v), got):
            y = y.double().cpu().numpy()
            rows = slice(batch.starts[0], batch.starts[-1])
            codes = oa.rows(x[rows].double().numpy().reshape(-1, dim), fmt)
            value = oa.row_values(*codes, fmt, dim).reshape(-1, heads, dim)
            assert np.array_equal(y[rows], value)
            assert (y[: batch.starts[0]] == 7).all() and (y[batch.starts[-1]:] == 7).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties_extremes_and_values_that_are_not_finite(fmt):
    import torch
    batch = Batch([(16, 16)], 16)
    x = torch.zeros(16, 2, 64)
    x[0, 0, :8] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[1, 0, 0], x[1, 0, 1], x[1, 0, 40] = float("inf"), 3.0, 2.0
    x[2, 0, 0], x[2, 0, 33] = float("nan"), -1.0
    x[3, 0], x[3, 1] = 3.0e38, 1e-38
    x[4, 0] = torch.linspace(-2, 2, 64) * 1e-41
    x[5, 0, ::7], x[5, 1, 5] = 2.0**-126, -2.0**127
    x[6, 0, 0], x[6, 0, 63] = 2688.0, 2.0**-9
    x[7, 0, 16:32], x[7, 0, 0] = 2.0**-20, 1.0
    cache = marked(batch, 2, 64, fmt)
    ddg.mx4_cache_append(cache, x.cuda(), (-x).cuda(), *batch.dev)
    want = expect(cache, batch, x.double().numpy(), -x.double().numpy(), fmt)
    nan = 255 if fmt == "mxfp4" else 127
    got = [t.cpu().numpy().view(np.uint8) for t in (cache.codes, cache.scales, cache.exponents)]
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[2], want[2])
    sound = np.repeat(want[1] != nan, want[0].shape[-1] // want[1].shape[-1], axis=-1)  # codes of a NaN block may be any
    assert np.array_equal(unsigned_zeros(got[0][sound]), unsigned_zeros(want[0][sound]))
    k, v = ddg.mx4_cache_read(cache, 16, *batch.dev, dtype=torch.float32)
    value = oa.row_values(*oa.rows(x.double().numpy().reshape(-1, 64), fmt), fmt, 64).reshape(16, 2, 64)
    assert np.array_equal(k.double().cpu().numpy(), value, equal_nan=True)
    assert np.array_equal(v.double().cpu().numpy(), -value, equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ("float32", "bfloat16"))
@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("dim,part", ((128, 128), (96, 24), (64, 6), (40, 40)))
def test_rotated_keys_are_rounded_once(fmt, dtype, interleaved, dim, part):
    """Codes of the 64-bit rotation rounded to 32 bits.  The kernel's 32-bit values are those but for about one in 10^2
    (2^-8 of a last place before the rounding), off by one last place: rows where a neighbouring 32-bit value gives
    other bytes are left out, and they are few."""
    import torch
    batch = Batch([(70000, 37), (9, 9)], 1024, seed=1)
    g = torch.Generator().manual_seed(dim + part)
    k, v = (torch.randn(batch.tokens, 3, dim, generator=g).to(getattr(torch, dtype)) for _ in range(2))
    table = ddg.rotary_table(part, base=1e4, interleaved=interleaved, scale=1.1)
    cache = marked(batch, 3, dim, fmt)
    ddg.mx4_cache_append(cache, k.cuda(), v.cuda(), *batch.dev, rotary=table)
    p = np.concatenate([batch.positions(b) for b in range(2)])
    turned = oa.rotary(k.double().numpy(), p, [int(t) % (1 << 64) for t in table.turns.cpu()], 1.1, interleaved).astype(np.float32)
    def shifted(to):  # the elements that are turned; the rest is copied exactly
        x = turned.copy()
        x[..., :part] = np.nextafter(x[..., :part], np.float32(to))
        return x

    near = [oa.rows(x.reshape(-1, dim), fmt) for x in (turned, shifted(np.inf), shifted(-np.inf))]
    firm = np.logical_and.reduce([(near[0][i] == other[i]).reshape(len(turned) * 3, -1).all(1) for i in range(3) for other in near[1:]]).reshape(-1, 3)
    assert firm.mean() > 0.99
    want = expect(cache, batch, turned.astype(np.float64), v.double().numpy(), fmt)
    got = [t.cpu().numpy().view(np.uint8) for t in (cache.codes, cache.scales, cache.exponents)]
    for b in range(2):
        for i, pos in enumerate(batch.positions(b)):
            page, off = batch.place(b, pos)
            for a, w in zip(got, want):
                ok = firm[batch.starts[b] + i]
                assert np.array_equal(a[page, 0, ok, off], w[page, 0, ok, off]) and np.array_equal(a[page, 1, :, off], w[page, 1, :, off])


@pytest.mark.parametrize("fmt", FORMATS)
def test_tokens_without_a_place(fmt):
    """Pages outside the cache, positions beyond the table and negative ones: not written, read as NaN."""
    import torch
    batch = Batch([(40, 40), (3, 5), (100, 70), (20, 4)], 16, table_pad=0)
    batch.table[0, 1], batch.table[3, 1] = batch.pages, -7
    batch.table = np.ascontiguousarray(batch.table[:, :5])  # the third sequence needs 7
    batch.dev[2] = torch.from_numpy(batch.table).cuda()
    k, v = (torch.randn(batch.tokens, 2, 64) for _ in range(2))
    cache = marked(batch, 2, 64, fmt)
    ddg.mx4_cache_append(cache, k.cuda(), v.cuda(), *batch.dev)
    same(cache, expect(cache, batch, k.double().numpy(), v.double().numpy(), fmt))
    got = torch.stack(ddg.mx4_cache_read(cache, batch.tokens, *batch.dev)).cpu()
    lost = np.zeros(batch.tokens, dtype=bool)
    for b in range(4):
        p = batch.positions(b)
        at = np.where((p < 0) | (p // 16 >= 5), -1, batch.table[b, np.clip(p // 16, 0, 4)])
        lost[batch.starts[b]: batch.starts[b + 1]] = (at < 0) | (at >= batch.pages)
    assert lost.sum() == 16 + 2 + 20 + 4 and lost.any()
    assert torch.isnan(got[:, lost]).all() and torch.isfinite(got[:, ~lost]).all()


def test_views_of_one_product():
    """Keys and values as parts of a fused projection, heads outermost, unaligned rows; read into parts of one array."""
    import torch
    batch = Batch([(50, 7), (31, 31)], 16)
    T = batch.tokens
    fused = torch.randn(T, 10, 96).bfloat16().cuda()
    k, v = fused[:, 6:8], fused[:, 8:]
    plain, other = (marked(batch, 2, 96, "nvfp4") for _ in range(2))
    ddg.mx4_cache_append(plain, k.contiguous(), v.contiguous(), *batch.dev)
    ddg.mx4_cache_append(other, k, v, *batch.dev)
    assert torch.equal(plain.codes, other.codes) and torch.equal(plain.scales, other.scales) and torch.equal(plain.exponents, other.exponents)
    other = marked(batch, 2, 96, "nvfp4")
    odd = torch.zeros(T * 2 * 97 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, 2, 97)[..., :96]
    odd.copy_(k)
    ddg.mx4_cache_append(other, odd, v.transpose(0, 1).contiguous().transpose(0, 1), *batch.dev)
    assert torch.equal(plain.codes, other.codes)
    both = torch.zeros(T, 4, 96, dtype=torch.float16, device="cuda")
    ddg.mx4_cache_read(plain, T, *batch.dev, out=(both[:, :2], both[:, 2:]))
    want = ddg.mx4_cache_read(plain, T, *batch.dev, dtype=torch.float16)
    assert torch.equal(both, torch.cat(want, 1))


@pytest.mark.parametrize("tokens,batch_size", ((1, 1), (300, 300), (5000, 3)))
def test_many_sequences_and_many_tokens(tokens, batch_size):
    import torch
    n = tokens // batch_size
    batch = Batch([(n + b % 7, n) for b in range(batch_size - 1)] + [(tokens, tokens - n * (batch_size - 1))], 16, seed=2)
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(batch.tokens, 2, 64, generator=g).bfloat16() for _ in range(2))
    for fmt in FORMATS:
        cache = ddg.mx4_cache(batch.pages, 16, 2, 64, fmt)
        ddg.mx4_cache_append(cache, k.cuda(), v.cuda(), *batch.dev)
        for x, y in zip((k, v), ddg.mx4_cache_read(cache, batch.tokens, *batch.dev, dtype=torch.float32)):
            q = ddg.mx4_dequantize(ddg.mx4_quantize(x.reshape(-1, 64).cuda(), fmt), torch.float32)
            assert torch.equal(y.reshape(-1, 64), q)
