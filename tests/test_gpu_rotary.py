"""Rotary positions against 64 bits, and their gradient."""
import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from oracle import attention as oa

pytestmark = pytest.mark.gpu

UNIT = {"bfloat16": 2.0**-8, "float16": 2.0**-11, "float32": 2.0**-24}


def turns_of(table):
    return [int(t) % (1 << 64) for t in table.turns.cpu()]


def check(x, y, positions, table, inverse=False):
    """Half a step of the type, and of 32 bits: cos and sin, the factor, two products and a sum."""
    got = y.double().cpu().numpy()
    xs = x.double().cpu().numpy()
    want = oa.rotary(xs, positions.cpu().numpy(), turns_of(table), table.scale, table.interleaved, inverse)
    n = table.turns.numel()
    size = np.abs(xs).copy()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if table.interleaved else (slice(0, n), slice(n, 2 * n))
    size[..., i] = size[..., j] = (np.abs(xs[..., i]) + np.abs(xs[..., j])) * abs(table.scale)
    unit = UNIT[str(y.dtype)[6:]]
    bound = unit * np.abs(want) + (4 * 2.0**-24) * (1 + unit) * size + (2.0**-25 if y.dtype.itemsize == 2 else 2.0**-149)
    bound[..., 2 * n:] = 0
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("dtype", sorted(UNIT))
@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("tokens,heads,dim,part", ((1, 1, 2, 2), (1, 40, 128, 128), (5, 3, 80, 20), (37, 7, 64, 32), (300, 5, 96, 48), (1300, 9, 128, 128),
                                                   (700, 33, 256, 64), (2, 2, 7, 4), (3, 1, 64, 0)))
def test_rotation_and_its_gradient(dtype, interleaved, tokens, heads, dim, part):
    import torch
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, heads, dim, generator=g).to(getattr(torch, dtype)).cuda()
    for wide, far in ((torch.int32, 1 << 17), (torch.int64, 1 << 40)):
        p = torch.randint(-far, far, (tokens,), generator=g).to(wide).cuda()
        table = ddg.rotary_table(part, base=500000.0, interleaved=interleaved, scale=1.0 if far < 1 << 20 else 1.2079441541679836)
        check(x, ddg.rotary(x, p, table), p, table)
        check(x, ddg.rotary_backward(x, p, table), p, table, inverse=True)


def test_far_positions_keep_their_angles():
    """2^31 - 1 with the fastest and the slowest pairs, in 32-bit values: an angle off by 2^-24 turns would show."""
    import torch
    table = ddg.rotary_table(64, base=1e6)
    p = torch.tensor([0, 1, (1 << 31) - 1, 123456789, -1, -(1 << 31)], dtype=torch.int64).cuda()
    x = torch.ones(6, 1, 64).cuda()
    check(x, ddg.rotary(x, p, table), p, table)
    check(x, ddg.rotary(x, p.int(), table), p, table)


@pytest.mark.parametrize("dtype", ("bfloat16", "float32"))
@pytest.mark.parametrize("interleaved", (False, True))
def test_views_in_place_and_unaligned(dtype, interleaved):
    import torch
    T, H, D = 19, 6, 64
    table = ddg.rotary_table(32, interleaved=interleaved)
    p = torch.arange(T, dtype=torch.int32).cuda() * 77
    base = torch.randn(T, H + 4, D, generator=torch.Generator().manual_seed(3)).to(getattr(torch, dtype)).cuda()
    x = base[:, 2:2 + H]
    want = ddg.rotary(x.contiguous(), p, table)
    assert torch.equal(ddg.rotary(x, p, table), want)
    turned = torch.empty(H, T, D, dtype=x.dtype, device="cuda").transpose(0, 1)  # heads outermost
    assert ddg.rotary(x, p, table, out=turned) is turned and torch.equal(turned, want)
    odd = torch.zeros(T * H * (D + 1) + 1, dtype=x.dtype, device="cuda")[1:].view(T, H, D + 1)
    ddg.rotary(x, p, table, out=odd[..., :D])
    assert torch.equal(odd[..., :D], want) and not odd[..., D].any()
    copy = base.clone()
    ddg.rotary(copy[:, 2:2 + H], p, table, out=copy[:, 2:2 + H])
    assert torch.equal(copy[:, 2:2 + H], want) and torch.equal(copy[:, :2], base[:, :2]) and torch.equal(copy[:, 2 + H:], base[:, 2 + H:])
    with pytest.raises(ddg.DDGemmError):
        ddg.rotary(copy[:, 1:1 + H], p, table, out=copy[:, 2:2 + H])


def test_gradient_against_differences():
    """The map is linear: <rotary(x + h v) - rotary(x - h v), dy> / 2 h is <v, dx> but for the 32-bit roundings."""
    import torch
    g = torch.Generator().manual_seed(1)
    x, v, dy = (torch.randn(9, 4, 48, generator=g).cuda() for _ in range(3))
    p = torch.randint(0, 10000, (9,), generator=g).cuda()
    for interleaved in (False, True):
        table = ddg.rotary_table(40, interleaved=interleaved, scaling="bands", factor=4.0)
        ends = [(ddg.rotary(x + s * v, p, table).double() * dy.double()).sum() for s in (1.0, -1.0)]
        want = (v.double() * ddg.rotary_backward(dy, p, table).double()).sum()
        size = (v.abs().double() * dy.abs().double()).sum() + (x.abs().double() * dy.abs().double()).sum()
        assert abs((ends[0] - ends[1]) / 2 - want) <= 2 * table.scale * 8 * 2.0**-24 * size


def test_scalings():
    import math
    plain = ddg.rotary_table(64, base=10000.0)
    f = [t / 2.0**64 * 2 * math.pi for t in turns_of(plain)]
    assert all(abs(a / 10000.0 ** (-2 * i / 64) - 1) < 1e-12 for i, a in enumerate(f))
    linear = [t / 2.0**64 * 2 * math.pi for t in turns_of(ddg.rotary_table(64, scaling="linear", factor=4.0))]
    assert all(abs(a / b - 4) < 1e-12 for a, b in zip(f, linear))
    base = [t / 2.0**64 * 2 * math.pi for t in turns_of(ddg.rotary_table(64, scaling="base", factor=4.0))]
    assert abs(base[0] / f[0] - 1) < 1e-12 and abs(f[-1] / base[-1] - 4) < 1e-9  # the slowest pair by factor
    table = ddg.rotary_table(64, scaling="bands", factor=4.0, original=4096)
    bands = [t / 2.0**64 * 2 * math.pi for t in turns_of(table)]
    assert abs(bands[0] / f[0] - 1) < 1e-12 and abs(f[-1] / bands[-1] - 4) < 1e-12
    assert all(1 - 1e-12 <= a / b <= 4 + 1e-9 for a, b in zip(f, bands)) and abs(table.scale - (0.1 * math.log(4) + 1)) < 1e-15
    own = ddg.rotary_table(4, frequencies=[1.0, -0.25], scale=2.0)
    assert turns_of(own)[1] == (1 << 64) - int(0.25 / (2 * math.pi) * 2.0**64) and own.scale == 2.0


def test_no_tokens():
    import torch
    x = torch.zeros(0, 3, 16).cuda()
    assert ddg.rotary(x, torch.zeros(0, dtype=torch.int32).cuda(), ddg.rotary_table(16)).shape == (0, 3, 16)


@pytest.mark.parametrize("dtype", ("bfloat16", "float32"))
@pytest.mark.parametrize("interleaved", (False, True))
def test_the_widest_heads(dtype, interleaved):
    import torch
    x = torch.randn(1400, 2, 4096, generator=torch.Generator().manual_seed(0)).to(getattr(torch, dtype)).cuda()
    p = torch.arange(1400).cuda() * 3
    table = ddg.rotary_table(4096, interleaved=interleaved)
    y = ddg.rotary(x, p, table)
    check(x[::100], y[::100], p[::100], table)
