"""4-bit matrices and blocks whose offsets pass 32 bits: the far end of each
result equals that of the same rows by themselves."""
import pytest

import extended_precision_gemm_gb300 as ddg

pytestmark = pytest.mark.gpu


def test_quantised_matrix_beyond_32_bits():
    import torch
    rows, k = 70000, 32768  # 2.3e9 values
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda").normal_()
    for fmt in ("mxfp4", "nvfp4"):
        q = ddg.mx4_quantize(x, fmt)
        tail = x[-200:].contiguous()
        t = ddg.mx4_quantize(tail, fmt)
        assert torch.equal(q.codes[-200:], t.codes)
        v = ddg.mx4_dequantize(q)
        assert torch.equal(v[-200:], ddg.mx4_dequantize(t))
        del v
        # its columns: k of 70000, rows of 32768
        c = ddg.mx4_quantize(x, fmt, cols=True)
        part = ddg.mx4_quantize(x[:, -100:], fmt, cols=True)
        assert torch.equal(c.codes[-100:], part.codes)
        assert torch.equal(ddg.mx4_dequantize(c)[-100:], ddg.mx4_dequantize(part))
        del q, c
    torch.cuda.empty_cache()


def test_product_beyond_32_bits():
    import torch
    m, n, k = 70000, 32768, 128  # 2.3e9 outputs
    for fmt in ("mxfp4", "nvfp4"):
        a, b = (torch.empty(r, k, dtype=torch.bfloat16, device="cuda").normal_() for r in (m, n))
        qa, qb = ddg.mx4_quantize(a, fmt), ddg.mx4_quantize(b, fmt)
        C = ddg.mx4_gemm(qa, qb)
        # the same tiles of 256 rows: sums in the same order
        tail = ddg.mx4_gemm(ddg.mx4_quantize(a[-(m % 256) - 256:].contiguous(), fmt), qb)
        assert torch.equal(C[-(m % 256) - 256:], tail)
        del C
    torch.cuda.empty_cache()
    assert ddg.wait_timeouts() == 0


def test_block_beyond_32_bits():
    import torch
    T, D, F = 180000 - 180000 % 256, 64, 12288  # 2.2e9 hidden values
    w = [torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(std=0.1) for s in ((F, D), (F, D), (D, F))]
    x, dy = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    y, saved = ddg.ff_gated(x, *w, save=True)
    dx = ddg.ff_gated_backward(dy, x, *w, saved, need=(True, False, False, False))[0]
    del saved
    n = 8192
    y1, s1 = ddg.ff_gated(x[-n:], *w, save=True)
    dx1 = ddg.ff_gated_backward(dy[-n:], x[-n:], *w, s1, need=(True, False, False, False))[0]
    # tiles and their order along k may differ: a rounding of h and of the output
    for a, b in ((y, y1), (dx, dx1)):
        assert ((a[-n:].double() - b.double()).norm() <= 2.0**-8 * b.double().norm()).item()
    for fmt in ("mxfp4", "nvfp4"):
        q = ddg.mx4_ff_weights(*w, fmt)
        z, z1 = ddg.mx4_ff_gated(x, *q), ddg.mx4_ff_gated(x[-n:], *q)
        assert ((z[-n:].double() - z1.double()).norm() <= 2.0**-7 * z1.double().norm()).item()
        del z
    torch.cuda.empty_cache()
    assert ddg.wait_timeouts() == 0
