"""Attention over the 4-bit cache against 64 bits: lengths, head layouts, masks,
pages, strides, streams."""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import attention as oa

from attention_util import Batch, check, filled, queries

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp4", "nvfp4")
DTYPES = ("bfloat16", "float16")


def run(sizes, page, heads, group, dim, fmt, dtype, window=0, sinks=0, scale=None, seed=0, rows=None, **more):
    batch = Batch(sizes, page, seed=seed, **more)
    cache, values = filled(batch, heads, dim, fmt, seed, rows)
    q = queries(batch, heads * group, dim, dtype, seed)
    y = ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks, scale=scale)
    check(y, q, batch, values, dtype, window, sinks, scale)
    return batch, cache, values, q, y


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", (1, 8, 40, 64, 72, 96, 128, 200, 256))
def test_one_token_each(fmt, dtype, dim):
    run([(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (64, 1), (65, 1), (300, 1), (1025, 1)], 16, 2, 4, dim, fmt, dtype, seed=dim)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,group", ((1, 1), (3, 1), (1, 5), (2, 7), (1, 8), (2, 9), (1, 16), (1, 24), (1, 64), (8, 2)))
def test_head_layouts(fmt, heads, group):
    run([(100, 1), (37, 3), (260, 2)], 32, heads, group, 128, fmt, "bfloat16", seed=group)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,group", ((64, 4), (128, 1), (128, 4), (128, 8), (256, 3)))
def test_prompts_and_parts_of_them(fmt, dtype, dim, group):
    run([(5, 5), (0, 0), (129, 129), (400, 33), (64, 0), (700, 260), (1, 1)], 16, 2, group, dim, fmt, dtype, seed=group, lead=1, tail=2)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", ((1, 0), (1, 1), (7, 3), (16, 4), (100, 0), (100, 40), (1000, 4), (1 << 40, 5)))
def test_windows_and_sinks(fmt, window, sinks):
    run([(1, 1), (6, 1), (90, 1), (333, 4), (300, 200), (1200, 1)], 16, 2, 4, 64, fmt, "float16", window, sinks, seed=window % 97)


@pytest.mark.parametrize("page", (16, 64, 1024))
def test_long_sequences_cut_into_parts(page):
    run([(30011, 1)], page, 1, 8, 128, "nvfp4", "bfloat16")
    run([(9000, 1), (40, 1), (12345, 2)], page, 2, 4, 64, "mxfp4", "float16")
    run([(70001, 1)], page, 1, 1, 64, "mxfp4", "bfloat16", 5000, 30)


def test_more_new_tokens_than_tokens():
    """Queries at negative positions see nothing: zeros."""
    batch, _, _, _, y = run([(3, 7), (0, 4), (-5, 2), (20, 20)], 16, 2, 2, 64, "mxfp4", "bfloat16")
    assert not y[:4].any() and not y[7:13].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_very_different_sizes(fmt, dtype):
    """Keys and values over 2^+-30, and queries: references and exponents keep them in range."""
    rows = lambda rng, shape: 2.0 ** rng.integers(-30, 31, shape) * np.where(np.arange(shape[0]) == 0, 2.0**-28, 1.0).reshape(-1, 1, 1, 1)  # noqa: E731
    batch = Batch([(200, 1), (77, 20), (500, 3)], 16)
    cache, values = filled(batch, 2, 128, fmt, 5, rows)
    q = queries(batch, 8, 128, dtype)
    y = ddg.mx4_attention(q, cache, *batch.dev)
    y32 = y.double().cpu().numpy()
    for b in range(3):
        for h in range(8):
            at = slice(batch.starts[b], batch.starts[b + 1])
            want, size, most = oa.attention(q[at, h].double().cpu().numpy(), *values[b][:, h // 4], batch.positions(b), 128**-0.5)
            unit = 2.0**-8 if dtype == "bfloat16" else 2.0**-11
            with np.errstate(over="ignore"):
                far = np.abs(want) >= 65504 if dtype == "float16" else np.zeros_like(want, bool)
            err = (2 * 140 * 2.0**-23 * most + 2.0**-11)[:, None] * size
            assert (np.abs(y32[at, h] - want) <= unit * (np.abs(want) + err) + err + 2.0**-24)[~far].all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", (1, 3, 40, 150))
def test_what_is_not_seen_does_not_matter(fmt, n):
    """NaN in rows behind the sequence (the fill of every cache here), outside the window, and in
    tokens that only later queries see: those alone become NaN, in the blocks of values that are."""
    import torch
    length, window, sinks = 300, 100, 2
    batch = Batch([(length, n)], 16)
    cache, values = filled(batch, 1, 64, fmt)
    q = queries(batch, 4, 64, "bfloat16")
    nan = 255 if fmt == "mxfp4" else 127
    p = batch.positions(0)

    def spoil(j, kv, block):
        page, off = batch.place(0, j)
        cache.scales[page, kv, 0, off, block] = nan

    for j in (2, 50, int(p[0]) - window):  # neither a sink nor in any window
        spoil(j, 0, 0)
        spoil(j, 1, 1)
    for head in range(4):
        check(ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks), q, batch, values, "bfloat16", window, sinks)
    last = int(p[-1])
    spoil(last, 1, 1)
    y = ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks)
    size = 32 if fmt == "mxfp4" else 16
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[-1, :, size: 2 * size] = True
    assert torch.equal(torch.isnan(y), bad)
    if n > 2:
        spoil(last - 1, 0, 0)  # a key: every element of the two rows that see it
        y = ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks)
        bad[-2:] = True
        assert torch.equal(torch.isnan(y), bad)
        spoil(int(p[0]) - window + 1, 1, 0)  # seen by the first query alone
        y = ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks)
        bad[0, :, :size] = True
        assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("n", (1, 40, 200))
def test_pages_that_are_not_there(n):
    """The queries that see them are NaN, the others what they are without."""
    import torch
    batch = Batch([(250, n), (40, 1)], 16, table_pad=0)
    cache, values = filled(batch, 2, 64, "nvfp4")
    q = queries(batch, 8, 64, "bfloat16")
    want = ddg.mx4_attention(q, cache, *batch.dev)
    for bad in (-1, batch.pages, 1 << 30):
        table = batch.dev[2].clone()
        table[0, 14] = bad  # tokens 224 .. 239
        y = ddg.mx4_attention(q, cache, *batch.dev[:2], table)
        hit = torch.from_numpy(np.concatenate([batch.positions(0) >= 224, [False]]))
        assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], want[~hit])
    y = ddg.mx4_attention(q, cache, *batch.dev[:2], batch.dev[2][:, :10].contiguous())  # a table of 160 tokens
    hit = torch.from_numpy(np.concatenate([batch.positions(0) >= 160, [False]]))
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], want[~hit])
    lengths = batch.dev[1].clone()
    lengths[0] = (1 << 31) - 1
    y = ddg.mx4_attention(q, cache, batch.dev[0], lengths, batch.dev[2])
    assert torch.isnan(y[:n]).all() and torch.equal(y[n:], want[n:])


@pytest.mark.parametrize("n", (1, 50))
def test_strides_and_rows_of_no_sequence(n):
    import torch
    batch = Batch([(120, n), (77, n)], 16, lead=3, tail=4)
    cache, values = filled(batch, 2, 96, "mxfp4")
    fused = torch.randn(batch.tokens, 12, 96, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q = fused[:, :8]
    out = torch.full((8, batch.tokens, 96), 5.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert ddg.mx4_attention(q, cache, *batch.dev, out=out) is out
    check(out, q, batch, values, "bfloat16")
    assert (out[:3] == 5).all() and (out[-4:] == 5).all()
    odd = torch.zeros(batch.tokens * 8 * 97 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(batch.tokens, 8, 97)
    odd[..., :96] = q
    again = torch.zeros_like(odd)
    ddg.mx4_attention(odd[..., :96], cache, *batch.dev, out=again[..., :96])
    assert torch.equal(again[3:-4, :, :96], out[3:-4]) and not again[..., 96].any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_cache_beyond_32_bit_offsets(fmt):
    """Over 2^32 bytes of codes, the sequence's pages at its ends."""
    import torch
    page, heads, dim = 1024, 8, 256
    small = Batch([(2100, 2)], page, spare=0, table_pad=0)
    cache, values = filled(small, heads, dim, fmt)
    pages = (1 << 32) // (2 * heads * page * dim // 2) + 40
    big = ddg.mx4_cache(pages, page, heads, dim, fmt)
    at = torch.tensor([pages - 1, 0, pages - 2])
    order = torch.from_numpy(small.table[0]).long()
    for a, b in ((big.codes, cache.codes), (big.scales, cache.scales), (big.exponents, cache.exponents)):
        a[at.cuda()] = b[order.cuda()]
    table = at.int().view(1, 3).cuda()
    q = queries(small, 16, dim, "bfloat16")
    y = ddg.mx4_attention(q, big, *small.dev[:2], table)
    check(y, q, small, values, "bfloat16")
    k, v = ddg.mx4_cache_read(big, 2, *small.dev[:2], table, dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy().astype(np.float64).transpose(1, 0, 2), values[0][0][:, -2:])
    ddg.mx4_cache_append(big, k * 2, v, *small.dev[:2], table)
    k2, _ = ddg.mx4_cache_read(big, 2, *small.dev[:2], table, dtype=torch.float32)
    assert torch.equal(k2, k * 2)


def test_streams_and_graphs():
    """On a side stream, captured and replayed with other inputs, and two graphs at once."""
    import torch
    batch = Batch([(5000, 1), (300, 1), (4, 3), (900, 80)], 16)
    cache, values = filled(batch, 2, 64, "mxfp4")
    table = ddg.rotary_table(64)
    q = queries(batch, 8, 64, "bfloat16")
    k, v = (torch.randn(batch.tokens, 2, 64, device="cuda").bfloat16() for _ in range(2))
    p = torch.from_numpy(np.concatenate([batch.positions(b) for b in range(4)])).cuda()

    def step(q, k, v, stream=None):
        ddg.mx4_cache_append(cache, k, v, *batch.dev, rotary=table, stream=stream)
        return ddg.mx4_attention(ddg.rotary(q, p, table, stream=stream), cache, *batch.dev, stream=stream)

    want = step(q, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(q, k, v, side)
    side.synchronize()
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ddg.mx4_attention(ddg.rotary(q, p, table), cache, *batch.dev))
        graphs.append(g)
    for seed in range(3):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)))
        want = ddg.mx4_attention(ddg.rotary(q, p, table), cache, *batch.dev)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_equal_calls_give_equal_bits():
    import torch
    batch = Batch([(20000, 1), (77, 60), (3, 1)], 64)
    cache, _ = filled(batch, 2, 128, "nvfp4")
    q = queries(batch, 16, 128, "float16")
    first = ddg.mx4_attention(q, cache, *batch.dev)
    for _ in range(5):
        assert torch.equal(ddg.mx4_attention(q, cache, *batch.dev), first)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,group", ((64, 4), (128, 2)))
def test_a_prompt_and_then_token_by_token(fmt, dim, group):
    """Rotation, append and attention as a program runs them, against the whole thing in 64 bits on what the cache holds."""
    import torch
    heads, page, prompt, steps = 2, 16, 75, 20
    lengths = [prompt, 9]
    batch = Batch([(n + steps, 0) for n in lengths], page, table_pad=0)
    cache = ddg.mx4_cache(batch.pages, page, heads, dim, fmt)
    table = ddg.rotary_table(dim, base=1e4)
    pages = batch.dev[2]
    keys, vals, qs, ys = ([[], []] for _ in range(4))
    g = torch.Generator().manual_seed(3)
    done = [0, 0]
    for step in range(steps + 1):
        new = lengths if step == 0 else [1, 1]
        T = sum(new)
        qkv = torch.randn(T, heads * (group + 2), dim, generator=g).bfloat16().cuda()
        q, k, v = qkv.split([heads * group, heads, heads], 1)
        done = [a + n for a, n in zip(done, new)]
        starts = torch.tensor([0, new[0], T], dtype=torch.int32).cuda()
        now = torch.tensor(done, dtype=torch.int32).cuda()
        p = torch.cat([torch.arange(d - n, d) for d, n in zip(done, new)]).cuda()
        ddg.mx4_cache_append(cache, k, v, starts, now, pages, rotary=table)
        ddg.rotary(q, p, table, out=q)
        y = ddg.mx4_attention(q, cache, starts, now, pages)
        for b, at in enumerate((slice(0, new[0]), slice(new[0], T))):
            keys[b].append(k[at]), vals[b].append(v[at]), qs[b].append(q[at]), ys[b].append(y[at])
    starts = torch.tensor([0, done[0], sum(done)], dtype=torch.int32).cuda()
    now = torch.tensor(done, dtype=torch.int32).cuda()
    kk, vv = ddg.mx4_cache_read(cache, sum(done), starts, now, pages, dtype=torch.float32)
    whole = Batch([(n, n) for n in done], page)
    values = [torch.stack((kk, vv))[:, a:e].permute(0, 2, 1, 3).double().cpu().numpy() for a, e in ((0, done[0]), (done[0], sum(done)))]
    q = torch.cat([torch.cat(x) for x in qs])
    check(torch.cat([torch.cat(x) for x in ys]), q, whole, values, "bfloat16")
    # the keys are those of the rotation to the 4-bit format's rounding (a sixth of a block's largest value for mxfp4's codes)
    k64 = np.concatenate([oa.rotary(torch.cat(keys[b]).double().cpu().numpy(), np.arange(done[b]), [int(t) % (1 << 64) for t in table.turns.cpu()]) for b in range(2)])
    most = np.abs(k64).reshape(*k64.shape[:2], -1, 16 if fmt == "nvfp4" else 32).max(-1).repeat(16 if fmt == "nvfp4" else 32, -1)
    assert (np.abs(kk.cpu().numpy() - k64) <= most * (0.26 if fmt == "mxfp4" else 0.2)).all()
    assert np.array_equal(vv.cpu().numpy(), ddg.mx4_dequantize(ddg.mx4_quantize(torch.cat([torch.cat(x) for x in vals]).reshape(-1, dim), fmt), torch.float32).cpu().numpy().reshape(vv.shape))


def test_no_wait_gave_up():
    """After the calls above (the count is of the process)."""
    assert ddg.wait_timeouts() == 0


def test_the_first_call_on_a_cold_cache():
    """Loads from memory, not from L2: the last tile's values arrive long after its weights."""
    import torch
    batch = Batch([(129, 129), (700, 260)], 16)
    cache, values = filled(batch, 2, 256, "nvfp4")
    q = queries(batch, 6, 256, "float16")
    other = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    want = ddg.mx4_attention(q, cache, *batch.dev)
    check(want, q, batch, values, "float16")
    for i in range(5):
        other.fill_(i)
        assert torch.equal(ddg.mx4_attention(q, cache, *batch.dev), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,n", ((96, 1), (96, 40), (32, 1), (32, 40), (30, 2), (200, 1), (200, 40), (130, 30)))
def test_what_lies_beyond_the_head_does_not_matter(fmt, dtype, dim, n):
    """Rows are filled up to 64, 128 or 256 elements: any bytes there, NaN scales among them, leave the result as it is."""
    import torch
    batch = Batch([(200, n), (77, n), (n, n)], 16)
    cache, values = filled(batch, 2, dim, fmt)
    q = queries(batch, 6, dim, dtype)
    want = ddg.mx4_attention(q, cache, *batch.dev)
    check(want, q, batch, values, dtype)
    size = 32 if fmt == "mxfp4" else 16
    first = -(-dim // size)  # the first block beyond the head
    g = torch.Generator().manual_seed(0)
    for byte in (255, 127, 254, 0):
        cache.scales[..., first:] = byte
        spoilt = torch.randint(0, 256, cache.codes.shape, generator=g, dtype=torch.uint8).cuda()
        cache.codes[..., first * size // 2:] = spoilt[..., first * size // 2:]
        assert torch.equal(ddg.mx4_attention(q, cache, *batch.dev), want)
    k, _ = ddg.mx4_cache_read(cache, batch.tokens, *batch.dev, dtype=torch.float32)
    assert torch.isfinite(k).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", (-0.1, 0.0, 3.0))
@pytest.mark.parametrize("n", (1, 60))
def test_scales_of_either_sign(fmt, scale, n):
    run([(90, n), (200, n)], 16, 2, 4, 64, fmt, "bfloat16", scale=scale, seed=3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (1, 60))
def test_queries_that_are_not_finite_spoil_their_own_rows_only(dtype, n):
    import torch
    batch = Batch([(90, n), (200, n)], 16)
    cache, values = filled(batch, 2, 64, "nvfp4")
    q = queries(batch, 8, 64, dtype)
    want = ddg.mx4_attention(q, cache, *batch.dev)
    q[0, 1, 3], q[n, 2, 5] = float("nan"), float("inf")
    y = ddg.mx4_attention(q, cache, *batch.dev)
    bad = torch.zeros(y.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[n, 2] = True
    assert torch.isnan(y[0, 1]).all()  # NaN scores
    assert not torch.isfinite(y[n, 2]).all()  # scores of plus infinity: NaN weights, as of the definition
    assert torch.equal(y[~bad], want[~bad])


def test_queries_of_any_size():
    """Rows of 2^-100 to 2^60: scaled into the range of 16 bits by a power of two."""
    import torch
    batch = Batch([(90, 1), (200, 60)], 16)
    cache, values = filled(batch, 1, 128, "mxfp4", 0, lambda rng, shape: 2.0**-20 * np.ones(shape))
    q = queries(batch, 4, 128, "bfloat16")
    powers = torch.tensor([-100, -60, 0, 60], device="cuda").float()
    for scale in (1.0, 2.0**-50):
        big = (q.double() * torch.exp2(powers.double())[None, :, None]).bfloat16()
        small = (q.double() * torch.exp2(powers.double())[None, :, None] * scale).bfloat16()
        y = ddg.mx4_attention(small, cache, *batch.dev, scale=2.0**-40 / scale)
        assert torch.equal(y, ddg.mx4_attention(big, cache, *batch.dev, scale=2.0**-40))
        check(y, big, batch, values, "bfloat16", scale=2.0**-40)


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_and_short_parts_in_one_batch(fmt):
    """Single tokens, some tokens and long parts together: each sequence takes the kernel that suits it."""
    sizes = [(200 + 7 * b, 1) for b in range(40)] + [(900, 600)] + [(100 + b, 3) for b in range(30)] + [(300, 150), (64, 13)] + [(33, 1)] * 60
    run(sizes, 16, 2, 4, 64, fmt, "float16", seed=1, lead=2, tail=3)
    run(sizes, 16, 1, 8, 128, fmt, "bfloat16", 50, 3, seed=2)


def test_an_empty_cache():
    import torch
    cache = ddg.mx4_cache(0, 16, 2, 64, "mxfp4")
    for n in (1, 100):
        starts, lengths = torch.tensor([0, n, n + 2], dtype=torch.int32).cuda(), torch.tensor([n, 0], dtype=torch.int32).cuda()
        table = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
        x = torch.randn(n + 2, 2, 64, device="cuda").bfloat16()
        ddg.mx4_cache_append(cache, x, x, starts, lengths, table)
        y = ddg.mx4_attention(x, cache, starts, lengths, table)
        assert torch.isnan(y[:n]).all() and not y[n:].any()
        k, v = ddg.mx4_cache_read(cache, n + 2, starts, lengths, table)
        assert torch.isnan(k).all() and torch.isnan(v).all()


def test_no_tokens_and_no_sequences():
    import torch
    cache = ddg.mx4_cache(4, 16, 2, 64, "nvfp4")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    ddg.mx4_attention(q, cache, torch.zeros(1, dtype=torch.int32, device="cuda"), none, none.view(0, 4), out=out)
    assert (out == 5).all()
    assert ddg.mx4_attention(q[:0], cache, torch.zeros(2, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"),
                             torch.zeros(1, 4, dtype=torch.int32, device="cuda")).shape == (0, 4, 64)


def test_calls_on_two_streams_at_once():
    import torch
    batch = Batch([(6000, 1), (300, 1), (4, 3), (2000, 300)], 16)
    cache, values = filled(batch, 2, 128, "mxfp4")
    q = queries(batch, 8, 128, "bfloat16")
    few = Batch([(3000, 1), (77, 2)], 16)
    cache2, _ = filled(few, 4, 64, "nvfp4")
    q2 = queries(few, 16, 64, "float16")
    want, want2 = ddg.mx4_attention(q, cache, *batch.dev), ddg.mx4_attention(q2, cache2, *few.dev)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        got = [(ddg.mx4_attention(q, cache, *batch.dev, stream=a), ddg.mx4_attention(q2, cache2, *few.dev, stream=b)) for _ in range(5)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) and torch.equal(y, want2) for x, y in got)


@pytest.mark.parametrize("n", (1, 60))
def test_windows_and_sinks_beyond_every_position(n):
    import torch
    batch = Batch([(90, n), (200, n)], 16)
    cache, _ = filled(batch, 2, 64, "mxfp4")
    q = queries(batch, 4, 64, "bfloat16")
    want = ddg.mx4_attention(q, cache, *batch.dev)
    for window, sinks in ((2**31 - 65536, 0), (2**31 - 65537, 3), (2**62, 1), (5, 2**40), (5, 2**31 - 65537), (2**31 - 65537, 2**31 - 65537)):
        assert torch.equal(ddg.mx4_attention(q, cache, *batch.dev, window=window, sinks=sinks), want), (window, sinks)


def test_a_long_part_among_many_single_tokens():
    """More sequences than the long parts' rows could be of: their tiles are numbered by tokens."""
    sizes = [(30 + b % 50, 1) for b in range(300)] + [(400, 333)] + [(20 + b, 1) for b in range(200)] + [(260, 7), (90, 6), (150, 150)]
    run(sizes, 16, 2, 8, 64, "nvfp4", "bfloat16", seed=4)
    run(sizes, 16, 1, 1, 128, "mxfp4", "float16", 40, 2, seed=5, lead=3, tail=5)


@pytest.mark.parametrize("fmt,dim", (("mxfp4", 64), ("nvfp4", 128), ("mxfp4", 256)))
def test_a_page_table_for_far_more_than_there_is(fmt, dim):
    """How many parts a row has goes by its own sequence: none, one, some and the most of them."""
    import torch
    sizes = [(0, 0), (70, 70), (511, 100), (513, 90), (1100, 130), (2600, 70), (40, 60)]
    for window, sinks in ((0, 0), (600, 20)):
        batch, cache, values, q, y = run(sizes, 16, 1, 2, dim, fmt, "bfloat16", window, sinks, seed=6, lead=1, tail=2)
        starts, lengths, table = batch.dev
        wide = torch.nn.functional.pad(table, (0, 2000), value=-1)
        z = ddg.mx4_attention(q, cache, starts, lengths, wide, window=window, sinks=sinks)
        check(z, q, batch, values, "bfloat16", window, sinks)
