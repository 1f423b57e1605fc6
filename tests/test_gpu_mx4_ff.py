"""The gated block on 4-bit operands against 64 bits.

The weights' and x's 4-bit values are exact (test_gpu_mx4.py), so g, u and h
differ from the exact ones by the 32-bit sums and the activation (the bounds of
test_gpu_ff.py).  Quantising h then takes either the exact path's code and
scale, or, where h or the largest of its block lies within that error of an
edge, a neighbour's: the bound spans the codes and scales of h - e and h + e.
"""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import microscaled as ms

pytestmark = pytest.mark.gpu

UNIT = {"bfloat16": 2.0**-8, "float16": 2.0**-11, "float32": 2.0**-24}


def _torch():
    import torch
    return torch


def hidden_span(h, e, fmt):
    """(quantised h, largest deviation of what h +- e quantises to), (rows, F)."""
    F = h.shape[1]
    size = ms.BLOCK[fmt]
    blocks = lambda t: np.pad(t, ((0, 0), (0, -F % size))).reshape(t.shape[0], -1, size)  # noqa: E731
    code, byte, exps = ms.quantize(h, fmt)
    value = ms.values(code, byte, exps, fmt, F)
    sign = np.sign(h)
    variants = [np.maximum(np.abs(h) - e, 0), np.abs(h), np.abs(h) + e]
    worst = np.zeros_like(h)
    for scaled in variants:
        _, byte, exps = ms.quantize(scaled, fmt)
        if fmt == "mxfp4":
            unit = np.ldexp(1.0, byte.astype(np.int64) - 127)
        else:
            unit = ms.e4m3_grid()[byte] * np.ldexp(1.0, exps)[:, None]
        unit = np.where(unit > 0, unit, 1.0)[..., None]
        for t in variants:
            v = (ms.CODES[ms.nearest_code(blocks(t), unit)] * unit).reshape(h.shape[0], -1)[:, :F] * sign
            worst = np.maximum(worst, np.abs(v - value))
    return value, worst


def check_block(T, D, F, fmt, dtype, act, seed):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, D, generator=g) * torch.exp(0.5 * torch.randn(1, D, generator=g))).to(getattr(torch, dtype)).cuda()
    wg, wu, wd = (torch.randn(r, c, generator=g).mul(c**-0.5).cuda() for r, c in ((F, D), (F, D), (D, F)))
    w_in, w_out = ddg.mx4_ff_weights(wg, wu, wd, fmt)
    y = ddg.mx4_ff_gated(x, w_in, w_out, act=act)
    assert y.dtype == x.dtype and y.shape == (T, D)
    xv = ddg.mx4_dequantize(ddg.mx4_quantize(x, fmt), torch.float32).double()
    both = ddg.mx4_dequantize(w_in, torch.float32).double().view(-1, 2, 32, D)
    vg, vu = (both[:, i].reshape(-1, D)[:F] for i in range(2))
    vd = ddg.mx4_dequantize(w_out, torch.float32).double()
    assert torch.equal(vg, ddg.mx4_dequantize(ddg.mx4_quantize(wg, fmt), torch.float32).double())
    c = lambda K: (K / 16 + 8) * 2.0**-23  # noqa: E731
    gg, uu = xv @ vg.t(), xv @ vu.t()
    eg, eu = c(D) * (xv.abs() @ vg.abs().t()), c(D) * (xv.abs() @ vu.abs().t())
    a = torch.from_numpy(ms.activation(gg.cpu().numpy(), act)[0]).cuda()
    h = a * uu
    ea = 1.13 * eg + 2.0**-19 * gg.abs()
    eh = (uu.abs() + eu) * ea + a.abs() * eu + 2.0**-23 * h.abs()
    q, dq = (torch.from_numpy(t).cuda() for t in hidden_span(h.cpu().numpy(), eh.cpu().numpy(), fmt))
    want = q @ vd.t()
    bound = dq @ vd.abs().t() + c(F) * ((q.abs() + dq) @ vd.abs().t())
    bound = bound + UNIT[dtype] * (want.abs() + bound) + 2.0**-24
    worst = ((y.double() - want).abs() / bound).max().item()
    assert worst <= 1.0, worst
    # few codes lie near an edge: the whole stays close
    assert (y.double() - want).norm() <= (2 * UNIT[dtype] + 0.02) * want.norm() + 1e-12
    assert ddg.wait_timeouts() == 0


@pytest.mark.parametrize("fmt", ("mxfp4", "nvfp4"))
@pytest.mark.parametrize("T,D,F", [(1, 64, 32), (1, 256, 96), (1, 520, 1000), (2, 100, 77), (8, 1024, 640), (16, 64, 2048), (33, 300, 257),
                                   (64, 512, 511), (65, 128, 200), (130, 257, 320), (300, 640, 1100)])
def test_block_against_64_bits(T, D, F, fmt):
    i = T + D + F
    check_block(T, D, F, fmt, ("bfloat16", "float16", "float32")[i % 3], ("silu", "gelu", "gelu_tanh", "relu")[i % 4], i)


@pytest.mark.parametrize("act", ("silu", "gelu", "gelu_tanh", "relu"))
@pytest.mark.parametrize("T", (1, 260))
def test_every_activation(T, act):
    for fmt in ("mxfp4", "nvfp4"):
        check_block(T, 192, 288, fmt, "bfloat16", act, 5)


def test_strided_input_output_and_empty_sizes():
    torch = _torch()
    for fmt in ("mxfp4", "nvfp4"):
        for T in (3, 150):
            wg, wu, wd = (torch.randn(s, device="cuda") for s in ((72, 40), (72, 40), (40, 72)))
            w = ddg.mx4_ff_weights(wg, wu, wd, fmt)
            x = torch.randn(T, 45, device="cuda").bfloat16()
            out = torch.full((T, 51), 3.0, device="cuda", dtype=torch.bfloat16)
            y = ddg.mx4_ff_gated(x[:, 3:43], *w, out=out[:, 7:47])
            assert torch.equal(y, ddg.mx4_ff_gated(x[:, 3:43].contiguous(), *w))
            assert (out[:, :7] == 3).all() and (out[:, 47:] == 3).all()
        assert ddg.mx4_ff_gated(x[:0, 3:43], *w).shape == (0, 40)
        none = ddg.mx4_ff_weights(wg[:0], wu[:0], wd[:, :0], fmt)
        assert not ddg.mx4_ff_gated(x[:, 3:43], *none).any()


def test_repeated_calls_and_other_streams_agree():
    torch = _torch()
    for fmt in ("mxfp4", "nvfp4"):
        for T in (1, 40, 300):
            w = ddg.mx4_ff_weights(*(torch.randn(s, device="cuda") for s in ((416, 256), (416, 256), (256, 416))), fmt)
            x = torch.randn(T, 256, device="cuda").bfloat16()
            first = ddg.mx4_ff_gated(x, *w)
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            second = ddg.mx4_ff_gated(x, *w, stream=side)
            side.synchronize()
            assert torch.equal(first, second) and torch.equal(first, ddg.mx4_ff_gated(x, *w))


@pytest.mark.parametrize("fmt", ("mxfp4", "nvfp4"))
@pytest.mark.parametrize("T", (3, 150))
def test_rows_that_fill_up_the_last_group_take_no_part(T, fmt):
    """Whatever the rows beyond F hold, NaN among it, the outputs are the same."""
    torch = _torch()
    D, F = 96, 72
    w_in, w_out = ddg.mx4_ff_weights(*(torch.randn(s, device="cuda") for s in ((F, D), (F, D), (D, F))), fmt)
    x = torch.randn(T, D, device="cuda").bfloat16()
    want = ddg.mx4_ff_gated(x, w_in, w_out)
    blocks = -(-D // ms.BLOCK[fmt])
    rows = [g * 64 + h * 32 + i for g in (2,) for h in (0, 1) for i in range(F - 64, 32)]
    at = [ms.scale_offset(r, b, fmt, D) for r in rows for b in range(blocks)]
    w_in.scales[torch.tensor(at, device="cuda")] = 255 if fmt == "mxfp4" else 127
    w_in.codes[torch.tensor(rows, device="cuda")] = 0x55
    assert torch.equal(ddg.mx4_ff_gated(x, w_in, w_out), want)


@pytest.mark.parametrize("T", (2, 140))
def test_hidden_blocks_far_below_the_row(T):
    """nvfp4 blocks of hidden values 2^-4 to 2^-40 of the row's largest: scales
    that are normal, subnormal and the least one.  Below 2^-14.8 a value may be
    off by a further step of its block, at most 2^-18 of the row's largest (the
    scale's least bit is 2^-9 2^e, max > 1344 2^e, and codes are at most 2
    apart); relu and powers of two keep everything else exact."""
    torch = _torch()
    D, F = 64, 320
    rng = np.random.default_rng(7)
    pick = lambda *s: rng.choice([-1.0, 1.0, 2.0, 0.5], s)  # noqa: E731
    small = np.repeat(2.0 ** -np.array([0, 4, 9, 13, 14, 15, 17, 19, 24, 40] * 2)[: F // 16], 16)
    wg, wu, wd = pick(F, D) / 8, pick(F, D) / 8 * small[:, None], pick(D, F)
    x = pick(T, D)
    t = [torch.from_numpy(v).float().cuda() for v in (x, wg, wu, wd)]
    w_in, w_out = ddg.mx4_ff_weights(*t[1:], "nvfp4")
    y = ddg.mx4_ff_gated(t[0], w_in, w_out, act="relu").double().cpu().numpy()
    both = ddg.mx4_dequantize(w_in, torch.float32).double().cpu().numpy().reshape(-1, 2, 32, D)
    vg, vu = both[:, 0].reshape(-1, D)[:F], both[:, 1].reshape(-1, D)[:F]
    vd = ddg.mx4_dequantize(w_out, torch.float32).double().cpu().numpy()
    xv = ddg.mx4_dequantize(ddg.mx4_quantize(t[0], "nvfp4"), torch.float32).double().cpu().numpy()
    h = np.maximum(xv @ vg.T, 0) * (xv @ vu.T)
    e = 2.0**-20 * (np.abs(xv) @ np.abs(vg).T) * (np.abs(xv) @ np.abs(vu).T)
    q, worst = hidden_span(h, e, "nvfp4")
    top = np.abs(h).max(axis=1, keepdims=True)
    assert ((np.abs(h) < 2.0**-15 * top) & (h != 0)).any()
    worst = worst + np.where(np.abs(h) < 2.0**-14 * top, 2.0**-18 * top, 0.0)
    want = q @ vd.T
    room = worst @ np.abs(vd).T + 2.0**-18 * (np.abs(q) @ np.abs(vd).T)
    assert (np.abs(y - want) <= room).all(), (np.abs(y - want) / room).max()


@pytest.mark.parametrize("fmt", ("mxfp4", "nvfp4"))
@pytest.mark.parametrize("T,D,F", [(2433, 64, 160), (3001, 96, 8200)])
def test_many_tokens(T, D, F, fmt):
    check_block(T, D, F, fmt, "bfloat16", "silu", T)


def test_hidden_blocks_far_below_the_row_for_many_tokens():
    test_hidden_blocks_far_below_the_row(2600)
