"""Attention over the 4-bit cache where scores, keys and values are far from one:
large scores, rows and blocks of very different sizes."""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import attention as oa

from attention_bounds import UNIT
from attention_util import Batch, filled, queries

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp4", "nvfp4")
DTYPES = ("bfloat16", "float16")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,dim", (([(90, 1), (200, 1)], 64), ([(300, 3)], 256), ([(9001, 1)], 128)))
def test_scores_of_any_size(fmt, dtype, sizes, dim):
    """Where one score is further above the others than they are off by, its token's value is the answer, whatever the
    scores' size: 2^x counts lifts and exponents of rows beside them."""
    batch = Batch(sizes, 16)
    cache, values = filled(batch, 1, dim, fmt, 2, lambda rng, shape: 2.0 ** rng.integers(-5, 6, shape))
    q = queries(batch, 2, dim, dtype)
    qn = q.double().cpu().numpy()
    for power in (5, 15, 20, 22, 24, 27, 30, 40, 60):
        for sign in (1.0, -1.0):
            y = ddg.mx4_attention(q, cache, *batch.dev, scale=sign * 2.0**power).double().cpu().numpy()
            alone = 0
            for b in range(len(sizes)):
                k, v = values[b][:, 0]
                for i, p in enumerate(batch.positions(b)):
                    s, size = sign * qn[batch.starts[b] + i] @ k[: p + 1].T, np.abs(qn[batch.starts[b] + i]) @ np.abs(k[: p + 1]).T
                    low, top = np.sort(s, 1)[:, -2:].T
                    # e^-30 of the others in all, and what both scores are off by (as in attention_bounds)
                    sure = (top - low) * 2.0**power > 30 + np.log(p + 1) + 2.0**power * 2 * size.max(1) * ((dim + 12) * 2.0**-23 + 2.0**-24)
                    want = v[s.argmax(1)]
                    got = y[batch.starts[b] + i]
                    assert np.isfinite(got).all(), (power, b, i)
                    off = np.abs(got - want) - (UNIT[dtype] + 2.0**-19) * np.abs(want) - 2.0**-12 * np.abs(v[: p + 1]).max() * np.exp(-30) - 2.0**-24 * (dtype == "float16")
                    assert (off[sure] <= 0).all(), (power, sign, b, i)
                    alone += sure.sum()
            assert alone > 0.8 * batch.tokens * 2 or power < 15, (power, alone)


def test_no_wait_gave_up_in_these():
    assert ddg.wait_timeouts() == 0
