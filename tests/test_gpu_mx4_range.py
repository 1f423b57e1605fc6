"""Row exponents and factors of any size in nvfp4 matrices, such as those of
matrices quantised elsewhere: values and products are those of the definition,
infinite or zero only where it leaves the type's range."""
import pytest

import extended_precision_gemm_gb300 as ddg
from tests.test_gpu_mx4 import sample

pytestmark = pytest.mark.gpu

EXPONENTS = [0, -126, 126, -127, 127, -140, 140, 165, -165, 200, -250, 1000, -1000, 2**31 - 1, -(2**31)]
LEAST = {"float32": 2.0**-149, "bfloat16": 2.0**-133, "float16": 2.0**-24}
MOST = {"float32": (2 - 2.0**-23) * 2.0**127, "bfloat16": (2 - 2.0**-7) * 2.0**127, "float16": 65504.0}
UNIT = {"float32": 2.0**-24, "bfloat16": 2.0**-8, "float16": 2.0**-11}


def _torch():
    import torch
    return torch


def matrix(rows, k, exponents, seed):
    """(a matrix with these row exponents, codes times scales in 64 bits, its exponents)."""
    torch = _torch()
    q = ddg.mx4_quantize(torch.from_numpy(sample(rows, k, seed, 0.5)).float().cuda(), "nvfp4")
    e = [exponents[i % len(exponents)] for i in range(rows)]
    plain = ddg.MX4(q.codes, q.scales, torch.zeros_like(q.exponents), rows, k, "nvfp4")
    base = ddg.mx4_dequantize(plain, torch.float32).double()
    q = ddg.MX4(q.codes, q.scales, torch.tensor(e, dtype=torch.int32).cuda(), rows, k, "nvfp4")
    return q, base, torch.tensor(e, dtype=torch.float64).cuda()


def times_power(v, e):
    """v 2^e, e bounded to +-900, which leaves the range of every type and none of 64 bits."""
    torch = _torch()
    e = e.clamp(-900, 900)
    for _ in range(8):
        v = v * torch.exp2((e / 8).floor())
    return v * torch.exp2(e - 8 * (e / 8).floor())


def check(got, want, bound, dtype):
    torch = _torch()
    got = got.double()
    most = MOST[dtype]
    inside, outside = want.abs() + bound < most, want.abs() - bound > most * (1 + UNIT[dtype])
    assert got[inside].isfinite().all()
    assert ((got - want).abs() <= bound)[inside].all(), ((got - want).abs() / bound)[inside].max().item()
    assert torch.equal(got[outside], torch.sign(want[outside]) * float("inf"))
    assert (inside | outside).double().mean() > 0.99


@pytest.mark.parametrize("dtype", sorted(UNIT))
@pytest.mark.parametrize("rows,k", [(15, 96), (31, 1000)])
def test_values(rows, k, dtype):
    q, base, e = matrix(rows, k, EXPONENTS, rows)
    want = times_power(base, e[:, None])
    check(ddg.mx4_dequantize(q, getattr(_torch(), dtype)), want, UNIT[dtype] * want.abs() + LEAST[dtype], dtype)


@pytest.mark.parametrize("dtype", sorted(UNIT))
@pytest.mark.parametrize("M,N,K", [(15, 60, 96), (60, 130, 300), (150, 75, 96), (400, 660, 300)])
def test_products(M, N, K, dtype):
    a, va, e = matrix(M, K, EXPONENTS, M)
    b, vb, f = matrix(N, K, EXPONENTS[::-1] + [3], N)
    s = e[:, None] + f[None, :]
    want = times_power(va @ vb.t(), s)
    room = times_power((K / 16 + 8) * 2.0**-23 * (va.abs() @ vb.abs().t()), s)
    check(ddg.mx4_gemm(a, b, getattr(_torch(), dtype)), want, room + UNIT[dtype] * (want.abs() + room) + LEAST[dtype], dtype)
    assert ddg.wait_timeouts() == 0
