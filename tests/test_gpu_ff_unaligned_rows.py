"""Rows that are whole 16-byte pieces but not whole 128-byte lines, at token
counts below and above the one from which such operands are copied."""
import pytest

import extended_precision_gemm_gb300 as ddg
from tests.test_gpu_ff import check, expected, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("T", (2049, 6000, 6001))
@pytest.mark.parametrize("D,F", [(72, 136), (200, 264)])
def test_forward_and_gradients(T, D, F, dtype):
    x, wg, wu, wd, dy = inputs(T, D, F, dtype, T + D)
    want = expected(x, wg, wu, wd, dy, "silu", dtype)
    y, saved = ddg.ff_gated(x, wg, wu, wd, save=True)
    grads = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    check(dict(zip(("y", "dx", "dwg", "dwu", "dwd"), (y, *grads))), want, want)
