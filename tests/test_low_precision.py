"""The 4-bit formats' oracle against rational brute force, and the refusals of
the 4-bit and feed-forward entry points (no GPU needed)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import microscaled as ms


@pytest.fixture(scope="module")
def lib():
    return ddg.load()


# ---- the oracle ----

def brute_code(x, unit):
    """The nearest code by exact distances, ties to the even index."""
    r = abs(Fraction(x)) / unit
    best = sorted(range(8), key=lambda i: (abs(Fraction(ms.CODES[i]) - r), i % 2))
    return best[0]


@pytest.mark.parametrize("fmt", sorted(ms.BLOCK))
def test_oracle_rounds_to_the_nearest_code(fmt):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((6, 70)) * np.exp(2 * rng.standard_normal((6, 70)))).astype(np.float32)
    x[1, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    x[2] = 0
    code, byte, exps = ms.quantize(x, fmt)
    size = ms.BLOCK[fmt]
    for r in range(6):
        for k in range(70):
            b = k // size
            if fmt == "mxfp4":
                unit = Fraction(2) ** (int(byte[r, b]) - 127)
            else:
                unit = Fraction(float(ms.e4m3_grid()[byte[r, b]])) * Fraction(2) ** int(exps[r])
            if unit == 0:
                assert code[r, b, k % size] & 7 == 0
            else:
                assert code[r, b, k % size] & 7 == brute_code(float(x[r, k]), unit)


def test_oracle_scales():
    x = np.zeros((3, 32))
    x[0, 3], x[1, 3], x[2, 3] = 8.0, 7.99, 4.0
    assert ms.quantize(x, "mxfp4")[1].tolist() == [[128], [127], [127]]  # 4 <= max / scale < 8
    x = np.zeros((4, 16))
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 2688.0, 2689.0, 1344.0, 2688.0 * 2.0**-100
    _, byte, exps = ms.quantize(x, "nvfp4")
    assert exps.tolist() == [0, 1, -1, -100] and byte[0, 0] == byte[2, 0] == byte[3, 0] == 126
    for r in range(4):  # the nearest E4M3 number to max / (6 2^e)
        want = Fraction(float(x[r, 0])) / 6 / Fraction(2) ** int(exps[r])
        grid = [Fraction(float(v)) for v in ms.e4m3_grid()]
        assert byte[r, 0] == min(range(127), key=lambda i: (abs(grid[i] - want), i % 2))


def test_tile_scales_matches_the_layout():
    torch = pytest.importorskip("torch")
    for fmt, blocks in (("mxfp4", 9), ("nvfp4", 17)):
        s = torch.randint(0, 255, (200, blocks), dtype=torch.uint8)
        k = blocks * ms.BLOCK[fmt]
        t = ddg.mx4_tile_scales(s, fmt)
        assert t.numel() == ddg.mx4_layout(200, k, fmt)[1]
        for r in (0, 31, 32, 127, 128, 199):
            for b in (0, 3, 4, blocks - 1):
                assert t[ms.scale_offset(r, b, fmt, k)] == s[r, b]


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(2)
    x, wg, wu, wd, dy = (rng.standard_normal(s) for s in ((4, 5), (6, 5), (6, 5), (5, 6), (4, 5)))
    for act in ("silu", "gelu", "gelu_tanh"):
        g = ms.gated(x, wg, wu, wd, act, dy)
        args = [x, wg, wu, wd]
        for i, name in enumerate(("dx", "dwg", "dwu", "dwd")):
            v = rng.standard_normal(args[i].shape)
            ends = [(ms.gated(*[a + s * v if j == i else a for j, a in enumerate(args)], act) * dy).sum() for s in (1e-5, -1e-5)]
            assert abs((ends[0] - ends[1]) / 2e-5 - (g[name] * v).sum()) < 1e-6 * (1 + np.abs(g[name] * v).sum())


# ---- refusals ----

A, B, C, D_, E, F_, Y = (ctypes.c_void_p(i << 40) for i in range(1, 8))
ODD = ctypes.c_void_p((9 << 40) + 8)


def test_layout_and_quantise_refusals(lib):
    n = ctypes.c_int64()
    assert lib.dd_mx4_layout(0, 130, 300, ctypes.byref(n), None) == 0 and n.value == 160
    assert lib.dd_mx4_layout(1, 130, 300, None, ctypes.byref(n)) == 0 and n.value == 2 * 8 * 512
    assert lib.dd_mx4_layout(2, 4, 4, None, None) == 1                            # unknown format
    assert lib.dd_mx4_layout(0, -1, 4, None, None) == 1
    assert lib.dd_mx4_layout(0, 4, (1 << 22) + 1, None, None) == 2
    assert lib.dd_mx4_layout(0, (1 << 28) + 1, 4, None, None) == 2

    def quant(fmt=0, t=1, cols=0, rows=8, k=64, x=A, ldx=64, codes=B, ldq=32, scales=C, e=D_):
        return lib.dd_mx4_quantize(fmt, t, cols, rows, k, x, ldx, codes, ldq, scales, e, None)

    assert quant(fmt=5) == 1 and quant(t=3) == 1 and quant(cols=2) == 1
    assert quant(rows=-1) == 1 and quant(k=-1) == 1
    assert quant(ldx=63) == 1 and quant(cols=1, ldx=7) == 1
    assert quant(x=None) == 1 and quant(codes=None) == 1 and quant(scales=None) == 1
    assert quant(fmt=1, e=None) == 1                                              # nvfp4 needs exponents
    assert quant(ldq=16) == 1 and quant(ldq=40) == 1                              # too short, not a multiple of 16
    assert quant(codes=ODD) == 1 and quant(scales=ODD) == 1
    assert quant(x=ctypes.c_void_p((1 << 40) + 1)) == 1                           # not aligned to its elements
    assert quant(codes=A) == 1                                                    # result over the input
    assert quant(rows=0) == 0
    assert lib.dd_mx4_dequantize(0, 1, 8, 64, A, 32, B, None, C, 63, None) == 1
    assert lib.dd_mx4_dequantize(0, 1, 8, 64, A, 32, B, None, None, 64, None) == 1
    assert lib.dd_mx4_dequantize(0, 1, 8, 64, A, 32, B, None, A, 64, None) == 1
    assert lib.dd_mx4_dequantize(1, 1, 8, 64, A, 32, B, None, C, 64, None) == 1
    assert lib.dd_mx4_dequantize(0, 7, 8, 64, A, 32, B, None, C, 64, None) == 1


def test_product_refusals(lib):
    def gemm(fmt=0, m=8, n=8, k=64, a=A, lda=32, sa=B, ea=None, b=C, ldb=32, sb=D_, eb=None, t=1, c=E, ldc=8):
        return lib.dd_mx4_gemm(fmt, m, n, k, a, lda, sa, ea, b, ldb, sb, eb, 1.0, t, c, ldc, None)

    assert gemm(fmt=3) == 1 and gemm(t=9) == 1 and gemm(m=-1) == 1 and gemm(n=-1) == 1 and gemm(k=-1) == 1
    assert gemm(k=1 << 23) == 2
    assert gemm(ldc=7) == 1 and gemm(lda=16) == 1 and gemm(ldb=33) == 1
    assert gemm(a=None) == 1 and gemm(sb=None) == 1 and gemm(c=None) == 1
    assert gemm(a=ODD) == 1 and gemm(sb=ODD) == 1
    assert gemm(fmt=1) == 1 and gemm(fmt=1, ea=F_) == 1                           # nvfp4 needs both exponents
    assert gemm(c=A) == 1 and gemm(c=D_) == 1
    assert gemm(c=ctypes.c_void_p((5 << 40) + 1)) == 1
    assert gemm(m=0, a=None, sa=None, c=None) == 0 and gemm(n=0) == 0


def test_block_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.dd_ff_gated_saved_size(0, 4, 4, ctypes.byref(n)) == 1              # not a 16-bit type
    assert lib.dd_ff_gated_saved_size(1, 4, 4, None) == 1
    assert lib.dd_ff_gated_saved_size(1, 1 << 29, 4, ctypes.byref(n)) == 2
    assert lib.dd_ff_gated_saved_size(1, 5, 100, ctypes.byref(n)) == 0
    size = n.value

    def fwd(t=1, act=0, T=5, D=8, F=100, x=A, ldx=8, wg=B, ldwg=8, wu=C, ldwu=8, wd=D_, ldwd=100, y=E, ldy=8, s=F_, ns=None):
        return lib.dd_ff_gated(t, act, T, D, F, x, ldx, wg, ldwg, wu, ldwu, wd, ldwd, y, ldy, s, size if ns is None else ns, None)

    assert fwd(t=0) == 1 and fwd(act=4) == 1 and fwd(act=-1) == 1 and fwd(T=-1) == 1 and fwd(F=-1) == 1
    assert fwd(ldx=7) == 1 and fwd(ldwg=7) == 1 and fwd(ldwd=99) == 1 and fwd(ldy=7) == 1
    assert fwd(x=None) == 1 and fwd(wu=None) == 1 and fwd(wd=None) == 1 and fwd(y=None) == 1
    assert fwd(ns=size - 1) == 1 and fwd(s=ODD) == 1
    assert fwd(y=A) == 1 and fwd(s=A) == 1 and fwd(s=E) == 1                      # overlaps
    assert fwd(T=0, y=None) == 0

    def bwd(T=5, D=8, F=100, dy=A, x=B, wg=C, wu=D_, wd=E, s=F_, ns=size, dx=Y, dwg=None, dwu=None, dwd=None, lddx=8):
        return lib.dd_ff_gated_backward(1, T, D, F, dy, 8, x, 8, wg, 8, wu, 8, wd, 100, s, ns, dx, lddx, dwg, 8, dwu, 8, dwd, 100, None)

    assert bwd(dy=None) == 1 and bwd(x=None) == 1 and bwd(s=None) == 1 and bwd(ns=size - 256) == 1 and bwd(s=ODD) == 1
    assert bwd(lddx=7) == 1 and bwd(T=-2) == 1 and bwd(F=1 << 29) == 2
    assert bwd(dx=A) == 1 and bwd(dx=F_) == 1 and bwd(dwg=Y) == 1                 # over an input, saved, another output

    def serve(fmt=0, t=1, act=0, T=3, D=64, F=40, x=A, ldx=64, ci=B, ldi=32, si=C, co=D_, ldo=32, so=E, y=F_, ldy=64, ei=None, eo=None):
        return lib.dd_mx4_ff_gated(fmt, t, act, T, D, F, x, ldx, ci, ldi, si, ei, co, ldo, so, eo, y, ldy, None)

    assert serve(fmt=2) == 1 and serve(t=4) == 1 and serve(act=9) == 1 and serve(T=-1) == 1
    assert serve(ldx=63) == 1 and serve(ldi=16) == 1 and serve(ldo=16) == 1 and serve(ldy=1) == 1
    assert serve(x=None) == 1 and serve(ci=None) == 1 and serve(so=None) == 1 and serve(y=None) == 1
    assert serve(fmt=1) == 1 and serve(fmt=1, ei=Y) == 1
    assert serve(y=A) == 1 and serve(y=C) == 1
    assert serve(T=0) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 4)
    with pytest.raises(TypeError):
        ddg.mx4_quantize(x)                                # not on a GPU
    with pytest.raises(ValueError):
        ddg.mx4_quantize(x, "fp4")
    with pytest.raises(TypeError):
        ddg.ff_gated(x, x, x, x)
    with pytest.raises(ValueError):
        ddg.mx4_layout(4, 4, "int4")
    q = ddg.MX4(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8), None, 4, 4, "mxfp4")
    with pytest.raises(TypeError):
        ddg.mx4_gemm(q, q)                                 # host tensors
    with pytest.raises(ValueError):
        ddg.mx4_gemm(q, ddg.MX4(q.codes, q.scales, None, 4, 5, "mxfp4"))
    with pytest.raises(ddg.DDGemmError) as e:
        ddg.mx4_layout(-1, 4)
    assert e.value.status == 1


def test_packed_calls_are_the_same_entry_points(lib):
    """dd_call_packed refuses what the entry points refuse (each by an argument near its end), and unknown calls."""
    import struct
    assert lib.dd_call_packed(6, struct.pack("=12q", *[0] * 12)) == 1
    assert lib.dd_call_packed(-1, struct.pack("=12q", *[0] * 12)) == 1
    assert lib.dd_call_packed(0, None) == 1
    a = [i << 40 for i in range(1, 9)]
    quant = lambda e: struct.pack("=12q", 1, 1, 0, 8, 64, a[0], 64, a[1], 32, a[2], e, 0)  # noqa: E731
    assert lib.dd_call_packed(0, quant(0)) == 1                                   # nvfp4 without exponents
    assert lib.dd_call_packed(0, struct.pack("=12q", 1 << 40, 1, 0, 8, 64, a[0], 64, a[1], 32, a[2], a[3], 0)) == 1
    assert lib.dd_call_packed(1, struct.pack("=11q", 0, 1, 8, 64, a[0], 32, a[1], 0, a[2], 63, 0)) == 1
    gemm = lambda ldc: struct.pack("=12qd4q", 0, 8, 8, 64, a[0], 32, a[1], 0, a[2], 32, a[3], 0, 1.0, 1, a[4], ldc, 0)  # noqa: E731
    assert lib.dd_call_packed(2, gemm(7)) == 1
    assert lib.dd_call_packed(2, struct.pack("=12qd4q", 0, 0, 8, 64, 0, 32, 0, 0, 0, 32, 0, 0, 1.0, 1, 0, 8, 0)) == 0
    assert lib.dd_call_packed(3, struct.pack("=19q", 0, 1, 0, 3, 64, 40, a[0], 64, a[1], 32, a[2], 0, a[3], 32, a[4], 0, a[5], 63, 0)) == 1
    assert lib.dd_call_packed(4, struct.pack("=18q", 1, 0, 5, 8, 100, a[0], 8, a[1], 8, a[2], 8, a[3], 100, a[4], 8, a[5], 16, 0)) == 1
    back = [1, 5, 8, 100, a[0], 8, a[1], 8, a[2], 8, a[3], 8, a[4], 100, a[5], 1 << 20, 0, 8, 0, 8, 0, 8, a[0], 100, 0]
    assert lib.dd_call_packed(5, struct.pack("=25q", *back)) == 1                 # dWd over dy
