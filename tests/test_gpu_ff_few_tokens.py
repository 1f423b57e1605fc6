"""The 16-bit block at and below 16 tokens, where hidden values keep what their
rounding leaves, and just above: operands and outputs inside wider matrices,
gradients on their own, other streams."""
import itertools

import pytest

import extended_precision_gemm_gb300 as ddg
from tests.test_gpu_ff import check, expected, inputs

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dwg", "dwu", "dwd")
TOKENS = (1, 15, 16, 17)


def _torch():
    import torch
    return torch


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("T", TOKENS)
def test_strided_and_misaligned_operands_and_outputs(T, dtype):
    torch = _torch()
    D, F = 40, 72
    x, wg, wu, wd, dy = inputs(T, D, F, dtype, 4)
    y, saved = ddg.ff_gated(x, wg, wu, wd, save=True)
    grads = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)

    def inside(t, off, more):
        wide = torch.full((t.shape[0], t.shape[1] + more), 9.0, dtype=t.dtype, device="cuda")
        wide[:, off : off + t.shape[1]] = t
        return wide[:, off : off + t.shape[1]]

    for off, more in ((1, 3), (8, 16), (3, 5)):
        v = [inside(t, off, more) for t in (x, wg, wu, wd, dy)]
        out = inside(torch.zeros_like(x), off, more)
        y2, saved2 = ddg.ff_gated(*v[:4], save=True, out=out)
        outs = [inside(torch.zeros_like(t), off, more) for t in (x, wg, wu, wd)]
        g2 = ddg.ff_gated_backward(v[4], *v[:4], saved2, dx=outs[0], dWg=outs[1], dWu=outs[2], dWd=outs[3])
        assert torch.equal(y2, y)
        for a, b, o in zip(g2, grads, outs):
            assert torch.equal(a, b) and a.data_ptr() == o.data_ptr()
        for o in outs + [out]:  # nothing beside the outputs was touched
            wide = o._base
            assert (wide[:, :off] == 9).all() and (wide[:, off + o.shape[1] :] == 9).all()
    assert ddg.wait_timeouts() == 0


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("D,F", [(64, 96), (136, 1100)])
@pytest.mark.parametrize("T", TOKENS)
def test_every_choice_of_gradients(T, D, F, dtype):
    x, wg, wu, wd, dy = inputs(T, D, F, dtype, T + D)
    want = expected(x, wg, wu, wd, dy, "silu", dtype)
    _, saved = ddg.ff_gated(x, wg, wu, wd, save=True)
    for need in itertools.product((False, True), repeat=4):
        part = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved, need=need)
        assert [p is not None for p in part] == list(need)
        got = {n: p for n, p in zip(NAMES, part) if p is not None}
        check(got, want, got)


@pytest.mark.parametrize("T", TOKENS)
def test_other_streams_and_repeated_calls_agree(T):
    torch = _torch()
    x, wg, wu, wd, dy = inputs(T, 256, 384, "bfloat16", 3)
    torch.cuda.synchronize()

    def step(**kw):
        y, s = ddg.ff_gated(x, wg, wu, wd, save=True, **kw)
        return (y, *ddg.ff_gated_backward(dy, x, wg, wu, wd, s, **kw))

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    second = step(stream=side)
    with torch.cuda.stream(side):
        third = step()
    side.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)
