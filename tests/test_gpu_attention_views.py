"""Inputs and outputs that are parts of one array, with no element in common: heads side
by side, halves of heads, heads outermost.  Results are those of arrays of their own."""
import pytest

import extended_precision_gemm_gb300 as ddg

from attention_util import Batch, filled, queries

pytestmark = pytest.mark.gpu


def pairs(torch, T, H, D, dtype):
    """(first, second) parts of T x H x D in one array, and the array."""
    side = torch.zeros(T, 2 * H + 1, D, dtype=dtype, device="cuda")
    yield side[:, :H], side[:, H + 1 :], side
    yield side[:, H : 2 * H], side[:, :H], side
    halves = torch.zeros(T, H, 2, D, dtype=dtype, device="cuda")
    yield halves[:, :, 0], halves[:, :, 1], halves
    yield halves[:, :, 1], halves[:, :, 0], halves
    outer = torch.zeros(2 * H, T, D, dtype=dtype, device="cuda")
    yield outer[::2].transpose(0, 1), outer[1::2].transpose(0, 1), outer
    tokens = torch.zeros(2 * T, H, D, dtype=dtype, device="cuda")
    yield tokens[1::2], tokens[::2], tokens
    ragged = torch.zeros(T, 2 * H * D + 3, dtype=dtype, device="cuda")
    yield ragged[:, : H * D].view(T, H, D), ragged[:, H * D + 3 :].view(T, H, D), ragged


def check_apart(torch, whole, first, second, before, want):
    """`second` holds want, everything else is what it was."""
    assert torch.equal(second, want)
    now = whole.clone()
    second.copy_(torch.zeros_like(want))
    assert torch.equal(whole, before), "elements of the other parts"
    whole.copy_(now)


@pytest.mark.parametrize("dtype", ("bfloat16", "float32"))
@pytest.mark.parametrize("T,H,D", ((9, 4, 64), (1, 3, 64), (700, 2, 40), (5, 1, 128)))
def test_rotary(dtype, T, H, D):
    import torch
    table = ddg.rotary_table(D)
    p = torch.arange(T, device="cuda")
    for first, second, whole in pairs(torch, T, H, D, getattr(torch, dtype)):
        first.copy_(torch.randn(first.shape, generator=torch.Generator().manual_seed(1)))
        second.copy_(torch.zeros_like(second))
        before = whole.clone()
        want = ddg.rotary(first.clone(), p, table)
        assert ddg.rotary(first, p, table, out=second) is second
        check_apart(torch, whole, first, second, before, want)


@pytest.mark.parametrize("sizes", ([(50, 1), (33, 2)], [(300, 90), (70, 70)], [(40, 1)]))
@pytest.mark.parametrize("dim", (64, 72))
def test_attention(sizes, dim):
    import torch
    batch = Batch(sizes, 16)
    cache, _ = filled(batch, 2, dim, "nvfp4")
    q = queries(batch, 4, dim, "bfloat16")
    want = ddg.mx4_attention(q, cache, *batch.dev)
    for first, second, whole in pairs(torch, batch.tokens, 4, dim, torch.bfloat16):
        first.copy_(q)
        second.copy_(torch.zeros_like(second))
        before = whole.clone()
        assert ddg.mx4_attention(first, cache, *batch.dev, out=second) is second
        check_apart(torch, whole, first, second, before, want)


def test_cache_read():
    import torch
    batch = Batch([(50, 7), (31, 31)], 16)
    cache, _ = filled(batch, 2, 64, "mxfp4")
    k, v = ddg.mx4_cache_read(cache, batch.tokens, *batch.dev)
    for first, second, whole in pairs(torch, batch.tokens, 2, 64, torch.bfloat16):
        ddg.mx4_cache_read(cache, batch.tokens, *batch.dev, out=(first, second))
        assert torch.equal(first, k) and torch.equal(second, v)


def test_parts_with_elements_in_common_are_refused():
    import torch
    T, H, D = 9, 4, 64
    table, p = ddg.rotary_table(D), torch.arange(9, device="cuda")
    side = torch.zeros(T, 2 * H, D, device="cuda").bfloat16()
    halves = torch.zeros(T, H, 2 * D, device="cuda").bfloat16()
    tokens = torch.zeros(2 * T, H, D, device="cuda").bfloat16()
    for x, y in ((side[:, :H], side[:, H - 1 : -1]), (side[:, 1 : H + 1], side[:, :H]), (side[:, ::2], side[:, :H]), (halves[..., :D], halves[..., D - 1 : -1]),
                 (tokens[:T], tokens[1 : T + 1]), (tokens[::2], tokens[:T])):
        with pytest.raises(ddg.DDGemmError):
            ddg.rotary(x, p, table, out=y)
