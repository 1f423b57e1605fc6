"""Infinities in the operands of the 16-bit gated block, from one token on.

An output is a NaN, an infinity of one sign or finite as the definition says,
evaluated here in 64 bits: the number of tokens, and with it whether the hidden
values keep what their rounding leaves, makes no difference.
"""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import microscaled as ms
from tests.test_gpu_ff import inputs

pytestmark = pytest.mark.gpu

OPERANDS = ("x", "wg", "wu", "wd", "dy")


def product(a, b):
    """a b with every sum taken term by term."""
    return (a[:, :, None] * b[None, :, :]).sum(axis=1)


def definition(x, wg, wu, wd, dy, act):
    with np.errstate(all="ignore"):
        g, u = product(x, wg.T), product(x, wu.T)
        a, da = ms.activation(g, act)
        h, dh = a * u, product(dy, wd)
        dg, du = dh * (u * da), dh * a
        return {"y": product(h, wd.T), "dx": product(dg, wg) + product(du, wu), "dwg": product(dg.T, x),
                "dwu": product(du.T, x), "dwd": product(dy.T, h)}


def kind(v):
    """0 finite, 1 and -1 the infinities, 2 NaN."""
    return np.where(np.isnan(v), 2, np.where(np.isinf(v), np.sign(v), 0)).astype(int)


def check_kinds(got, want):
    for name, t in got.items():
        k, w = kind(t.double().cpu().numpy()), kind(want[name])
        assert np.array_equal(k, w), (name, np.argwhere(k != w)[:5].tolist(), int((k != w).sum()))
    assert ddg.wait_timeouts() == 0


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("act", ("silu", "relu"))
@pytest.mark.parametrize("where", OPERANDS)
@pytest.mark.parametrize("T", (1, 7, 16, 17))
def test_infinite_operands(T, where, act, dtype):
    D, F = 40, 72
    t = dict(zip(OPERANDS, inputs(T, D, F, dtype, T)))
    m = t[where]
    m[0, 3], m[-1, m.shape[1] - 2] = float("inf"), -float("inf")
    args = [t[n] for n in OPERANDS]
    want = definition(*(v.double().cpu().numpy() for v in args), act)
    assert kind(want["y"]).any() or kind(want["dwd"]).any()
    y, saved = ddg.ff_gated(*args[:4], act=act, save=True)
    grads = ddg.ff_gated_backward(args[4], *args[:4], saved)
    check_kinds(dict(zip(("y", "dx", "dwg", "dwu", "dwd"), (y, *grads))), want)
    alone = ddg.ff_gated_backward(args[4], *args[:4], saved, need=(True, False, False, False))
    others = ddg.ff_gated_backward(args[4], *args[:4], saved, need=(False, True, True, True))
    check_kinds(dict(zip(("dx", "dwg", "dwu", "dwd"), alone[:1] + others[1:])), want)


@pytest.mark.parametrize("T", (1, 16, 17))
def test_weights_gradients_of_rows_that_are_whole_sectors(T):
    """dWd has rows of 32 bytes' multiples here, and dWg not: both ways of storing them."""
    for D, F in ((36, 64), (64, 36)):
        x, wg, wu, wd, dy = inputs(T, D, F, "bfloat16", 3)
        dy[0, 5], x[T - 1, 2] = float("inf"), 0.0
        want = definition(*(v.double().cpu().numpy() for v in (x, wg, wu, wd, dy)), "silu")
        _, saved = ddg.ff_gated(x, wg, wu, wd, save=True)
        got = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved, need=(False, True, True, True))
        check_kinds(dict(zip(("dwg", "dwu", "dwd"), got[1:])), want)


@pytest.mark.parametrize("T", (3, 16, 17))
def test_hidden_values_beyond_float16(T):
    """Hidden values of one token that float16 does not hold are infinite; the other tokens' outputs do not see them."""
    x, wg, wu, wd, _ = inputs(T, 64, 96, "float16", 12)
    x[:] = x.clamp(-2, 2)
    clean = ddg.ff_gated(x, wg, wu, wd, act="relu")
    x[1] *= 500
    y = ddg.ff_gated(x, wg, wu, wd, act="relu")
    g, u = (x.double() @ w.double().t() for w in (wg, wu))
    h = g.clamp(min=0) * u
    assert (h[1].abs() > 65520).any()
    assert not y[1].isfinite().any()
    keep = [i for i in range(T) if i != 1]
    assert (y[keep] == clean[keep]).all() and y[keep].isfinite().all()
