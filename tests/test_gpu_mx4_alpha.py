"""Factors that undo the operands' powers of two: no partial product leaves the
range where the result does not."""
import pytest

import extended_precision_gemm_gb300 as ddg
from tests.test_gpu_mx4_range import UNIT, matrix, times_power

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ("float32", "bfloat16"))
@pytest.mark.parametrize("alpha,e,f", [(1.3 * 2.0**120, -70, -60), (-1.3 * 2.0**100, -90, -10), (1.5 * 2.0**-140, 90, 60),
                                       (1.3 * 2.0**-100, 40, 60), (2.0**-149, 100, 50), (-0.7, 30, -25), (0.0, 100, 90)])
@pytest.mark.parametrize("M,N,K", [(5, 60, 96), (150, 75, 96), (400, 660, 300)])
def test_large_and_small_factors(M, N, K, alpha, e, f, dtype):
    import torch
    a, va, ea = matrix(M, K, [e, e - 3, e + 1], M)
    b, vb, eb = matrix(N, K, [f, f + 2], N)
    alpha = torch.tensor(alpha, dtype=torch.float32).double().item()
    s = ea[:, None] + eb[None, :]
    want = times_power(alpha * (va @ vb.t()), s)
    room = times_power((K / 16 + 8) * 2.0**-23 * abs(alpha) * (va.abs() @ vb.abs().t()), s)
    got = ddg.mx4_gemm(a, b, getattr(torch, dtype), alpha=alpha).double()
    bound = room + UNIT[dtype] * (want.abs() + room) + 2.0**-133
    assert got.isfinite().all() and ((got - want).abs() <= bound).all()
    assert want.any() or alpha == 0.0


@pytest.mark.parametrize("alpha", (float("inf"), -float("inf"), float("nan")))
def test_factors_that_are_not_finite(alpha):
    import torch
    for M in (5, 150):
        a, va, _ = matrix(M, 96, [0], M)
        b, vb, _ = matrix(40, 96, [0], 40)
        got, want = ddg.mx4_gemm(a, b, torch.float32, alpha=alpha), (alpha * (va @ vb.t())).float()
        assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
