"""The gated feed-forward block on the GPU, forward and backward, against 64 bits.

Every output is held to an elementwise bound that follows the roundings of the
computation.  u: half a unit in the last place of the type (2^-8 bfloat16,
2^-11 float16).  c(K) = (K / 16 + 8) 2^-23: the 32-bit sum of K products, one
truncation allowed for every 16 of them.  Activations are 1.13-Lipschitz and
their derivatives 0.8-Lipschitz (relu's is off by 1 within the error of g
around 0); evaluating them costs at most 2^-19 of max(1, |g|).  a = act(g) and
b = u act'(g) are kept with at least 11 bits for the backward pass.
"""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import microscaled as ms

pytestmark = pytest.mark.gpu

UNIT = {"bfloat16": 2.0**-8, "float16": 2.0**-11}
KEPT = 2.0**-11


def _torch():
    import torch
    return torch


def inputs(T, D, F, dtype, seed):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    shape = lambda r, c, s: (torch.randn(r, c, generator=g) * s).to(getattr(torch, dtype))  # noqa: E731
    x = shape(T, D, 1.0) * torch.exp(0.5 * torch.randn(1, D, generator=g)).to(getattr(torch, dtype))
    return [t.cuda() for t in (x, shape(F, D, D**-0.5), shape(F, D, D**-0.5), shape(D, F, F**-0.5), shape(T, D, 1.0))]


def expected(x, wg, wu, wd, dy, act, dtype):
    """{name: (value, bound)} in 64 bits, on the GPU."""
    torch = _torch()
    u_ = UNIT[dtype]
    tiny = 2.0**-24 if dtype == "float16" else 0.0
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    T, D = x.shape
    F = wg.shape[0]
    c = lambda K: (K / 16 + 8) * 2.0**-23  # noqa: E731
    g, u = x @ wg.t(), x @ wu.t()
    dg_, du_ = c(D) * (x.abs() @ wg.abs().t()), c(D) * (x.abs() @ wu.abs().t())
    a, da = (torch.from_numpy(t).cuda() for t in ms.activation(g.cpu().numpy(), act))
    ea = 1.13 * dg_ + 2.0**-19 * g.abs()
    eda = 0.8 * dg_ + 2.0**-19 * g.abs().clamp(min=1) if act != "relu" else (g.abs() <= dg_).double()
    h = a * u
    eh = (u.abs() + du_) * ea + a.abs() * du_
    eh = eh + u_ * (h.abs() + eh) + tiny
    y = h @ wd.t()
    ey = eh @ wd.abs().t() + c(F) * ((h.abs() + eh) @ wd.abs().t())
    out = {"y": (y, ey)}
    dh = dy @ wd
    edh = c(D) * (dy.abs() @ wd.abs())
    b = u * da
    eb = (da.abs() + eda) * du_ + u.abs() * eda
    eb, ea = eb + KEPT * (b.abs() + eb), ea + KEPT * (a.abs() + ea)
    gg, gu = dh * b, dh * a
    egg, egu = (b.abs() + eb) * edh + dh.abs() * eb, (a.abs() + ea) * edh + dh.abs() * ea
    egg, egu = egg + u_ * (gg.abs() + egg) + tiny, egu + u_ * (gu.abs() + egu) + tiny
    mg, mu = gg.abs() + egg, gu.abs() + egu
    out["dx"] = (gg @ wg + gu @ wu, egg @ wg.abs() + egu @ wu.abs() + c(2 * F) * (mg @ wg.abs() + mu @ wu.abs()))
    out["dwg"] = (gg.t() @ x, egg.t() @ x.abs() + c(T) * (mg.t() @ x.abs()))
    out["dwu"] = (gu.t() @ x, egu.t() @ x.abs() + c(T) * (mu.t() @ x.abs()))
    out["dwd"] = (dy.t() @ h, dy.abs().t() @ eh + c(T) * (dy.abs().t() @ (h.abs() + eh)))
    return {n: (v, e + u_ * (v.abs() + e) + tiny + 1e-30) for n, (v, e) in out.items()}


def check(got, want, names):
    for n in names:
        value, bound = want[n]
        worst = ((got[n].double() - value).abs() / bound).max().item() if value.numel() else 0.0
        assert worst <= 1.0, (n, worst)
    assert ddg.wait_timeouts() == 0


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 264, 1000), (2, 100, 77), (7, 31, 33), (16, 256, 512), (45, 520, 264), (64, 128, 96),
          (96, 256, 640), (130, 72, 129), (257, 257, 255), (300, 512, 1032), (600, 136, 264)]


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("T,D,F", SHAPES)
def test_forward_and_gradients_within_the_bounds(T, D, F, dtype):
    act = ("silu", "gelu", "gelu_tanh", "relu")[(T + D + F) % 4]
    x, wg, wu, wd, dy = inputs(T, D, F, dtype, T + D + F)
    want = expected(x, wg, wu, wd, dy, act, dtype)
    y, saved = ddg.ff_gated(x, wg, wu, wd, act=act, save=True)
    only = ddg.ff_gated(x, wg, wu, wd, act=act)
    dx, dwg, dwu, dwd = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    check({"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}, want, want)
    check({"y": only}, want, ("y",))


@pytest.mark.parametrize("act", ("silu", "gelu", "gelu_tanh", "relu"))
@pytest.mark.parametrize("scale", (1e-3, 1.0, 40.0))
def test_activations_over_their_range(act, scale):
    x, wg, wu, wd, dy = inputs(64, 64, 192, "bfloat16", 9)
    wg = (wg * scale).contiguous()
    want = expected(x, wg, wu, wd, dy, act, "bfloat16")
    y, saved = ddg.ff_gated(x, wg, wu, wd, act=act, save=True)
    dx, dwg, dwu, dwd = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    check({"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}, want, want)


@pytest.mark.parametrize("act", ("silu", "gelu", "gelu_tanh"))
def test_gradients_against_differences(act):
    """The change of sum(dy * y) along a direction, by central differences of
    the formula in 64 bits, against the gradients' inner product with it."""
    torch = _torch()
    T, D, F = 40, 48, 72
    x, wg, wu, wd, dy = inputs(T, D, F, "float16", 21)
    want = expected(x, wg, wu, wd, dy, act, "float16")
    _, saved = ddg.ff_gated(x, wg, wu, wd, act=act, save=True)
    grads = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    at = [t.double().cpu().numpy() for t in (x, wg, wu, wd)]
    d = dy.double().cpu().numpy()
    rng = np.random.default_rng(5)
    for i, name in enumerate(("dx", "dwg", "dwu", "dwd")):
        v = rng.standard_normal(at[i].shape)
        step = 1e-4
        ends = []
        for s in (step, -step):
            moved = list(at)
            moved[i] = at[i] + s * v
            ends.append((ms.gated(*moved, act) * d).sum())
        slope = (ends[0] - ends[1]) / (2 * step)
        inner = (grads[i].double().cpu().numpy() * v).sum()
        # the outputs' bounds, and 1e-5 of the slope's size for the third derivative
        room = (want[name][1].cpu().numpy() * np.abs(v)).sum() + 1e-5 * (np.abs(want[name][0].cpu().numpy() * v)).sum()
        assert abs(inner - slope) <= room, (name, inner, slope, room)
        assert room < 0.2 * np.abs(want[name][0].cpu().numpy() * v).sum()


def test_strided_and_misaligned_operands_and_outputs():
    torch = _torch()
    T, D, F = 33, 40, 72
    x, wg, wu, wd, dy = inputs(T, D, F, "bfloat16", 4)
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


def test_parts_of_the_gradients_and_empty_sizes():
    torch = _torch()
    x, wg, wu, wd, dy = inputs(20, 64, 96, "bfloat16", 8)
    _, saved = ddg.ff_gated(x, wg, wu, wd, save=True)
    full = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    for i in range(4):
        need = tuple(j == i for j in range(4))
        part = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved, need=need)
        assert torch.equal(part[i], full[i]) and all(part[j] is None for j in range(4) if j != i)
    for T, D, F in ((0, 64, 96), (20, 64, 0), (20, 0, 96)):
        e = inputs(T, D, F, "float16", 1) if min(T, D, F) > 0 else [
            torch.randn(s, device="cuda").half() for s in ((T, D), (F, D), (F, D), (D, F), (T, D))]
        y, s = ddg.ff_gated(*e[:4], save=True)
        assert y.shape == (T, D) and not y.any()
        for grad, like in zip(ddg.ff_gated_backward(e[4], *e[:4], s), e):
            assert grad.shape == like.shape and not grad.any()


def test_other_streams_and_repeated_calls_agree():
    torch = _torch()
    x, wg, wu, wd, dy = inputs(70, 256, 384, "bfloat16", 3)
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


def test_infinities_reach_what_depends_on_them_only():
    torch = _torch()
    x, wg, wu, wd, _ = inputs(40, 64, 96, "bfloat16", 2)
    x[7, 3] = float("inf")
    y = ddg.ff_gated(x, wg, wu, wd)
    bad = ~torch.isfinite(y)
    assert bad[7].any()
    bad[7] = False
    assert not bad.any()


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("T,D,F", [(3000, 136, 70), (9, 72, 3000), (2100, 200, 2200), (2500, 77, 131), (130, 40, 4000)])
def test_few_tiles_and_deep_sums(T, D, F, dtype):
    """Gradients whose sums are shared by several blocks and added up afterwards."""
    x, wg, wu, wd, dy = inputs(T, D, F, dtype, T + F)
    want = expected(x, wg, wu, wd, dy, "silu", dtype)
    y, saved = ddg.ff_gated(x, wg, wu, wd, save=True)
    dx, dwg, dwu, dwd = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    got = {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}
    check(got, want, want)
    again = ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    assert all(_torch().equal(a, got[n]) for a, n in zip(again, ("dx", "dwg", "dwu", "dwd")))


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("T,D,F", [(1, 128, 640), (2, 64, 128), (4, 130, 192), (8, 120, 979), (16, 400, 222), (5, 2100, 4200)])
def test_few_tokens_are_rounded_once(T, D, F, dtype):
    """Of up to 16 tokens an intermediate value's rounding leaves 2^-8 of itself
    at most, kept in turn: errors are those of the outputs' own rounding, with
    room of a tenth for the backward pass's factors (kept to 2^-11) and for sums
    in 32 bits."""
    torch = _torch()
    g = torch.Generator().manual_seed(T * 1000 + F)
    make = lambda r, c, s=1.0: (torch.randn(r, c, generator=g) * s).to(getattr(torch, dtype)).cuda()  # noqa: E731
    x, dy, wg, wu, wd = make(T, D), make(T, D), make(F, D, D**-0.5), make(F, D, D**-0.5), make(D, F, F**-0.5)
    y, saved = ddg.ff_gated(x, wg, wu, wd, act="silu", save=True)
    assert torch.equal(y, ddg.ff_gated(x, wg, wu, wd, act="silu"))
    got = (y,) + ddg.ff_gated_backward(dy, x, wg, wu, wd, saved)
    X, DY, G, U, W = (t.double() for t in (x, dy, wg, wu, wd))
    gg, uu = X @ G.t(), X @ U.t()
    p = torch.sigmoid(gg)
    a, da = gg * p, p + gg * p * (1 - p)
    dh = DY @ W
    dg, du = dh * uu * da, dh * a
    want = ((a * uu) @ W.t(), dg @ G + du @ U, dg.t() @ X, du.t() @ X, DY.t() @ (a * uu))
    for o, w in zip(got, want):
        least = (w.to(o.dtype).double() - w).norm()
        assert (o.double() - w).norm() <= 1.1 * least, ((o.double() - w).norm() / least).item()
    assert ddg.wait_timeouts() == 0
