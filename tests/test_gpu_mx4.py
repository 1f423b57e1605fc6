"""4-bit microscaled matrices on the GPU: codes, scales and exponents equal to
the oracle's bit for bit; products within a bound derived from the 32-bit sums.

Bound of a product.  The operands are exact, so C differs from the sum of the
exact products by the roundings of the 32-bit sums and the final one.  The
tensor core adds 64 products to the accumulator in one instruction; allowing a
truncation (2^-23 of the partial sum, itself at most sum |a b|) for every 16 of
them, and 8 more for the epilogue, |dC| <= (K / 16 + 8) 2^-23 sum |a b| + u |C|
with u = 2^-8 (bfloat16), 2^-11 (float16), 2^-24 (float32).
"""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import microscaled as ms

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp4", "nvfp4")
UNIT = {"bfloat16": 2.0**-8, "float16": 2.0**-11, "float32": 2.0**-24}


def _torch():
    import torch
    return torch


def _dtype(name):
    return getattr(_torch(), name)


def sample(rows, k, seed, spread=2.0):
    """Values of unequal size, with zeros, whole zero blocks and a zero row."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * np.exp(spread * rng.standard_normal((rows, 1)) + 0.7 * rng.standard_normal((rows, k)))
    x[rng.random((rows, k)) < 0.05] = 0.0
    if rows > 2:
        x[rows // 2] = 0.0
        x[rows // 3, : k // 2] = 0.0
    return x


def stored_parts(q):
    """Codes (rows, padded k), scale bytes (rows, blocks) and exponents of an MX4 on the host."""
    codes = q.codes.cpu().numpy()
    code = np.stack((codes & 15, codes >> 4), 2).reshape(q.rows, -1)
    flat = q.scales.cpu().numpy()
    blocks = -(-q.k // 256) * (256 // ms.BLOCK[q.fmt])
    r, b = np.meshgrid(np.arange(q.rows), np.arange(blocks), indexing="ij")
    return code, flat[ms.scale_offset(r, b, q.fmt, q.k)], (q.exponents.cpu().numpy() if q.fmt == "nvfp4" else None)


def check_quantised(q, x):
    code, byte, exps = ms.quantize(x, q.fmt)
    got_code, got_byte, got_exps = stored_parts(q)
    blocks = byte.shape[1]
    assert np.array_equal(got_byte[:, :blocks], byte)
    assert not got_byte[:, blocks:].any()
    bad = np.repeat(byte == (255 if q.fmt == "mxfp4" else 127), ms.BLOCK[q.fmt], axis=1)[:, : q.k]
    want = code.reshape(q.rows, -1)[:, : q.k]
    have = got_code[:, : q.k]
    # the sign of a zero is free
    same = (want == have) | ((want & 7 == 0) & (have & 7 == 0)) | bad
    assert same.all(), np.argwhere(~same)[:5]
    width = -(-q.k // 32) * 32
    assert not (got_code[:, q.k : width] & 7).any()
    if q.fmt == "nvfp4":
        assert np.array_equal(got_exps, exps)
    return ms.values(code, byte, exps, q.fmt, q.k)


@pytest.mark.parametrize("cols", (False, True))
@pytest.mark.parametrize("dtype", ("bfloat16", "float16", "float32"))
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 32), (3, 31), (5, 257), (130, 96), (33, 1000), (200, 520), (2, 17000)])
def test_quantise_matches_the_definition(rows, k, fmt, dtype, cols):
    torch = _torch()
    x = torch.from_numpy(sample(rows, k, rows * 1000 + k)).to(_dtype(dtype))
    t = (x.t().contiguous() if cols else x).cuda()
    q = ddg.mx4_quantize(t, fmt, cols=cols)
    v = check_quantised(q, x.double().numpy())
    for out in ("bfloat16", "float32"):
        d = ddg.mx4_dequantize(q, _dtype(out)).double().cpu().numpy()
        assert np.array_equal(d, torch.from_numpy(v).to(_dtype(out)).double().numpy())


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantise_ties_subnormals_and_the_ends_of_the_range(fmt):
    torch = _torch()
    rng = np.random.default_rng(3)
    k = 512
    rows = []
    rows.append(np.resize([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0], k))          # every tie
    rows.append(np.resize([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], k) * 2.0**-60)
    rows.append(np.nextafter(np.resize([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], k).astype(np.float32), np.float32(9)))
    rows.append(np.nextafter(np.resize([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], k).astype(np.float32), np.float32(0)))
    rows.append(rng.standard_normal(k) * 2.0**-140)                                              # subnormal
    rows.append(np.full(k, 3.4e38) * rng.uniform(0.1, 1, k))                                     # near the largest
    rows.append(2.0 ** rng.integers(-120, 120, k))                                               # blocks far apart
    rows.append(np.where(np.arange(k) == 5, 2688.0, 2.0**-20))                                    # scale at its top, and below its least
    rows.append(np.where(np.arange(k) == 5, np.nextafter(np.float32(2688), np.float32(9999)), 1.0))
    # block maxima at and beside the ties of the E4M3 grid
    grid = ms.e4m3_grid()
    mids = (6 * (grid[1:] + grid[:-1]) / 2).astype(np.float32)
    x = np.zeros(k)
    x[:: 16] = mids[40 : 40 + 32]
    x[1] = 2688.0
    rows.append(x)
    rows.append(np.nextafter(x.astype(np.float32), np.float32(9999)) * (x > 0))
    x = np.stack(rows).astype(np.float32)
    for cols in (False, True):
        t = torch.from_numpy(x).cuda()
        q = ddg.mx4_quantize(t.t().contiguous() if cols else t, fmt, cols=cols)
        check_quantised(q, x)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cols", (False, True))
def test_infinities_and_nans_stay_in_their_blocks(fmt, cols):
    torch = _torch()
    x = sample(7, 300, 5)
    x[1, 40], x[2, 41], x[3, 299] = np.inf, np.nan, -np.inf
    x[4] = np.nan
    x32 = torch.from_numpy(x).float()
    q = ddg.mx4_quantize(x32.t().contiguous().cuda() if cols else x32.cuda(), fmt, cols=cols)
    v = check_quantised(q, x32.double().numpy())
    d = ddg.mx4_dequantize(q, torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(d), np.isnan(v)) and np.array_equal(np.nan_to_num(d), np.nan_to_num(v).astype(np.float32))


@pytest.mark.parametrize("dtype", ("bfloat16", "float16", "float32"))
@pytest.mark.parametrize("rows,k", [(128, 1024), (300, 2600), (257, 4099), (1030, 1300)])
def test_columns_with_blocks_far_apart(rows, k, dtype):
    torch = _torch()
    rng = np.random.default_rng(rows)
    x = sample(rows, k, rows) * np.repeat(2.0 ** -rng.integers(0, 24, (rows, -(-k // 16))), 16, axis=1)[:, :k]
    x[rng.integers(0, rows, 40), rng.integers(0, k, 40)] = np.tile([np.inf, -np.inf, np.nan, 0.0], 10)
    x = torch.from_numpy(x).to(_dtype(dtype))
    for fmt in FORMATS:
        q = ddg.mx4_quantize(x.t().contiguous().cuda(), fmt, cols=True)
        check_quantised(q, x.double().numpy())
        r = ddg.mx4_quantize(x.cuda(), fmt)
        v, w = (ddg.mx4_dequantize(t, torch.float32).nan_to_num(7e30) for t in (q, r))
        assert torch.equal(v, w)


def test_quantise_strided_and_misaligned_inputs():
    torch = _torch()
    base = torch.randn(70, 700, device="cuda").to(torch.bfloat16)
    for view in (base[:, 1:301], base[1::2, 8:264], base[:33, 3:4]):
        for fmt in FORMATS:
            for cols in (False, True):
                a, b = ddg.mx4_quantize(view, fmt, cols=cols), ddg.mx4_quantize(view.contiguous(), fmt, cols=cols)
                assert torch.equal(ddg.mx4_dequantize(a), ddg.mx4_dequantize(b))
    q = ddg.mx4_quantize(base[:, :100].contiguous(), "mxfp4")
    out = torch.full((70, 131), 7.0, device="cuda")
    ddg.mx4_dequantize(q, torch.float32, out=out[:, 5:105])
    assert torch.equal(out[:, 5:105], ddg.mx4_dequantize(q, torch.float32)) and (out[:, :5] == 7).all() and (out[:, 105:] == 7).all()


def product(m, n, k, fmt, dtype, seed, alpha=1.0):
    torch = _torch()
    a, b = sample(m, k, seed), sample(n, k, seed + 1)
    qa, qb = (ddg.mx4_quantize(torch.from_numpy(x).float().cuda(), fmt) for x in (a, b))
    va, vb = (ddg.mx4_dequantize(q, torch.float32).double() for q in (qa, qb))
    C = ddg.mx4_gemm(qa, qb, dtype=_dtype(dtype), alpha=alpha).double()
    want, mass = alpha * (va @ vb.t()), abs(alpha) * (va.abs() @ vb.abs().t())
    bound = (k / 16 + 8) * 2.0**-23 * mass + UNIT[dtype] * want.abs() + 1e-30
    if dtype == "float16":
        bound = bound + 2.0**-25  # its subnormals
        C, want, bound = (t[want.abs() < 6e4] for t in (C, want, bound))
    worst = ((C - want).abs() / bound).max().item() if C.numel() else 0.0
    assert worst <= 1.0, worst
    assert ddg.wait_timeouts() == 0


SHAPES = [(1, 1, 1), (1, 16, 64), (1, 200, 300), (2, 129, 256), (7, 192, 257), (16, 320, 1024), (33, 1000, 500),
          (64, 193, 2048), (65, 64, 64), (128, 384, 31), (129, 191, 4100), (255, 577, 768), (300, 200, 640), (513, 1030, 1300)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_within_the_bound(m, n, k, fmt):
    product(m, n, k, fmt, "float32", m + n + k)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("m,n,k", [(1, 300, 640), (3, 4097, 288), (48, 511, 1536), (300, 577, 1000), (1100, 900, 2304)])
def test_product_in_16_bits(m, n, k, dtype, fmt):
    product(m, n, k, fmt, dtype, m + n, alpha=0.37)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_of_small_whole_numbers_is_exact(fmt):
    """Codes times powers of two whose sums stay below 2^24: no rounding at all."""
    torch = _torch()
    rng = np.random.default_rng(11)
    for m, n, k in [(5, 40, 512), (300, 400, 1024)]:
        a, b = (torch.from_numpy(ms.CODES[rng.integers(0, 8, (r, k))] * rng.choice([-1.0, 1.0], (r, k))).float() for r in (m, n))
        a[:, ::16], b[:, ::16] = 6.0, -6.0  # every block's scale is 1 (mxfp4) or exact (nvfp4)
        qa, qb = ddg.mx4_quantize(a.cuda(), fmt), ddg.mx4_quantize(b.cuda(), fmt)
        assert torch.equal(ddg.mx4_dequantize(qa, torch.float32).cpu(), a)
        C = ddg.mx4_gemm(qa, qb, dtype=torch.float32).cpu()
        assert torch.equal(C.double(), a.double() @ b.double().t())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", (3, 300))
def test_each_scale_reaches_its_own_products(fmt, m):
    """One block of each row is not zero, at a place of its own: a scale taken from a wrong row, block or byte shows."""
    torch = _torch()
    k, n = 1024, 260
    size = ms.BLOCK[fmt]
    rng = np.random.default_rng(m)
    a, b = np.zeros((m, k)), 6.0 * np.ones((n, k)) * 2.0 ** rng.integers(-6, 7, (n, 1))  # max / 6 is a power of two
    for i in range(m):
        at = (i * 7) % (k // size) * size
        a[i, at : at + size] = 6.0 * 2.0 ** rng.integers(-5, 6)
    for j in range(n):
        b[j] *= np.repeat(2.0 ** rng.integers(-3, 4, k // size), size)
    qa, qb = (ddg.mx4_quantize(torch.from_numpy(x).float().cuda(), fmt) for x in (a, b))
    C = ddg.mx4_gemm(qa, qb, dtype=torch.float32).double().cpu().numpy()
    va, vb = (ddg.mx4_dequantize(q, torch.float32).double().cpu().numpy() for q in (qa, qb))
    assert np.array_equal(va, a) and np.array_equal(vb, b)
    assert np.array_equal(C, a @ b.T)


def test_nan_scales_reach_only_their_rows_and_columns():
    torch = _torch()
    for fmt in FORMATS:
        for m in (4, 200):
            a, b = (torch.from_numpy(sample(r, 300, r)).float() for r in (m, 130))
            a[2, 10], b[5, 299] = float("nan"), float("inf")
            C = ddg.mx4_gemm(ddg.mx4_quantize(a.cuda(), fmt), ddg.mx4_quantize(b.cuda(), fmt), dtype=torch.float32)
            bad = torch.isnan(C)
            assert bad[2].all() and bad[:, 5].all()
            bad[2], bad[:, 5] = False, False
            assert not bad.any()


def test_product_into_strided_output_and_empty_sums():
    torch = _torch()
    qa, qb = (ddg.mx4_quantize(torch.randn(r, 200, device="cuda"), "mxfp4") for r in (70, 90))
    want = ddg.mx4_gemm(qa, qb, dtype=torch.float32)
    out = torch.full((70, 133), 5.0, device="cuda")
    ddg.mx4_gemm(qa, qb, dtype=torch.float32, out=out[:, 3:93])
    assert torch.equal(out[:, 3:93], want) and (out[:, :3] == 5).all() and (out[:, 93:] == 5).all()
    # nothing to sum, nothing to write
    for fmt in FORMATS:
        e = ddg.mx4_quantize(torch.empty(6, 0, device="cuda"), fmt)
        assert not ddg.mx4_gemm(e, ddg.mx4_quantize(torch.empty(9, 0, device="cuda"), fmt)).any()
        z = ddg.mx4_quantize(torch.empty(0, 64, device="cuda"), fmt)
        assert ddg.mx4_gemm(z, ddg.mx4_quantize(torch.randn(9, 64, device="cuda"), fmt)).shape == (0, 9)


@pytest.mark.parametrize("dtype", ("bfloat16", "float16", "float32"))
@pytest.mark.parametrize("m,n", [(300, 601), (261, 514), (129, 96), (300, 33)])
def test_product_into_rows_of_every_alignment(m, n, dtype):
    torch = _torch()
    t = getattr(torch, dtype)
    qa, qb = (ddg.mx4_quantize(torch.randn(r, 320, device="cuda"), "nvfp4") for r in (m, n))
    want = ddg.mx4_gemm(qa, qb, dtype=t)
    for ld in (640, 648, 642, 641):  # rows of whole sectors, of 16 bytes, of words, of elements
        for first in (0, 1, 2, 8, 16):
            out = torch.full((m, ld), 5.0, dtype=t, device="cuda")
            ddg.mx4_gemm(qa, qb, out=out[:, first:first + n])
            assert torch.equal(out[:, first:first + n], want), (ld, first)
            assert (out[:, :first] == 5).all() and (out[:, first + n:] == 5).all(), (ld, first)


def test_operands_with_wide_rows_and_scales_quantised_elsewhere():
    torch = _torch()
    x = torch.randn(40, 512, device="cuda")
    for fmt in FORMATS:
        q = ddg.mx4_quantize(x, fmt)
        wide = torch.zeros(40, 512, dtype=torch.uint8, device="cuda")
        wide[:, :256] = q.codes
        blocks = 512 // ms.BLOCK[fmt]
        r, b = np.meshgrid(np.arange(40), np.arange(blocks), indexing="ij")
        plain = torch.from_numpy(q.scales.cpu().numpy()[ms.scale_offset(r, b, fmt, 512)]).cuda()
        p = ddg.MX4(wide[:, :256], ddg.mx4_tile_scales(plain, fmt), q.exponents, 40, 512, fmt)
        assert torch.equal(ddg.mx4_gemm(p, q), ddg.mx4_gemm(q, q))


def test_calls_on_another_stream_and_repeated_calls_agree():
    torch = _torch()
    x, w = torch.randn(200, 1000, device="cuda"), torch.randn(300, 1000, device="cuda")
    torch.cuda.synchronize()
    for fmt in FORMATS:
        first = ddg.mx4_gemm(ddg.mx4_quantize(x, fmt), ddg.mx4_quantize(w, fmt))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        second = ddg.mx4_gemm(ddg.mx4_quantize(x, fmt, stream=side), ddg.mx4_quantize(w, fmt, stream=side), stream=side)
        with torch.cuda.stream(side):
            third = ddg.mx4_gemm(ddg.mx4_quantize(x, fmt), ddg.mx4_quantize(w, fmt))
        side.synchronize()
        assert torch.equal(first, second) and torch.equal(first, third)
