"""gelu of negative arguments, where g (1 + erf(g / sqrt 2)) / 2 is far below g:
its error is one of the small result, not one of g."""
import math

import pytest

import extended_precision_gemm_gb300 as ddg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,least", [("bfloat16", -8.0), ("float16", -4.5)])
def test_small_results_are_accurate(dtype, least):
    """y = gelu(g) u - gelu(8) v with v near gelu(g) u / 8, one token for each g.

    gelu(8) is 8 in 32 bits, and of up to 16 tokens hidden values keep twice the
    type's bits, so y is what the error of gelu(g) u leaves of it: 2^-18 of it
    for gelu, a unit of the kept bits (2^-17 bfloat16, 2^-22 float16), 2^-21 for
    the other operations in 32 bits, and the rounding of y."""
    import torch
    type_ = getattr(torch, dtype)
    unit, kept = (2.0**-8, 2.0**-17) if dtype == "bfloat16" else (2.0**-11, 2.0**-22)
    g = torch.linspace(least, -0.5, 320).to(type_)
    exact = torch.tensor([v * 0.5 * math.erfc(-v / math.sqrt(2)) for v in g.double().tolist()], dtype=torch.float64)
    u = (1.0 / exact.abs()).to(type_)
    h = exact * u.double()
    v = (h / 8).to(type_)
    x = torch.stack((g, u, torch.full_like(g, 8.0), v), 1).cuda()
    unit_rows = torch.eye(4, dtype=type_, device="cuda")
    wg, wu = unit_rows[0::2].contiguous(), unit_rows[1::2].contiguous()
    wd = torch.zeros(4, 2, dtype=type_, device="cuda")
    wd[0, 0], wd[0, 1] = 1.0, -1.0
    y = torch.cat([ddg.ff_gated(x[i : i + 16], wg, wu, wd, act="gelu") for i in range(0, 320, 16)])[:, 0].double().cpu()
    left = h - 8 * v.double()
    bound = h.abs() * (2.0**-18 + kept + 2.0**-21) + unit * left.abs() + (2.0**-24 if dtype == "float16" else 0.0)
    worst = ((y - left).abs() / bound).max().item()
    assert worst <= 1.0, (worst, g[((y - left).abs() / bound).argmax()].item())
