"""The oracle of rotary positions, the 4-bit cache and attention over it against
closed forms, and what their entry points refuse (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import extended_precision_gemm_gb300 as ddg
from extended_precision_gemm_gb300 import attention as at
from extended_precision_gemm_gb300 import low_precision as lp
from oracle import attention as oa
from oracle import microscaled as ms


@pytest.fixture(scope="module")
def lib():
    return ddg.load()


# ---- the oracle ----

def test_rotation_is_the_multiplication_of_complex_numbers():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 2, 10))
    turns = [(1 << 64) // 7, 12345678901234567, (1 << 64) - 99]
    p = [0, 1, -3, 1000, 1 << 40, 7, 14]
    for interleaved in (False, True):
        y = oa.rotary(x, p, turns, 1.5, interleaved)
        for t in range(7):
            for i, turn in enumerate(turns):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
                z = (x[t, :, a] + 1j * x[t, :, b]) * 1.5 * np.exp(2j * np.pi * ((p[t] * turn) % (1 << 64) / 2.0**64))
                assert np.allclose(y[t, :, a], z.real, atol=1e-12) and np.allclose(y[t, :, b], z.imag, atol=1e-12)
        assert np.array_equal(y[..., 6:], x[..., 6:])
        back = oa.rotary(y, p, turns, 1 / 1.5, interleaved, inverse=True)
        assert np.allclose(back, x, atol=1e-12)
        # the gradient: <R x, dy> = <x, R^T dy>
        dy = rng.standard_normal(x.shape)
        assert abs((y * dy).sum() - (x * oa.rotary(dy, p, turns, 1.5, interleaved, inverse=True)).sum()) < 1e-10


def test_attention_of_equal_keys_is_the_mean():
    v = np.arange(12.0).reshape(6, 2)
    y, _, _ = oa.attention(np.ones((3, 2)), np.ones((6, 2)), v, [-1, 2, 5], 1.0)
    assert not y[0].any() and np.allclose(y[1], v[:3].mean(0)) and np.allclose(y[2], v.mean(0))
    y, _, _ = oa.attention(np.ones((1, 2)), np.ones((6, 2)), v, [5], 1.0, window=2, sinks=1)
    assert np.allclose(y[0], v[[0, 4, 5]].mean(0))


@pytest.mark.parametrize("fmt", sorted(ms.BLOCK))
def test_stored_rows_stand_for_the_quantised_values(fmt):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((20, 72)) * np.exp(3 * rng.standard_normal((20, 1)))).astype(np.float32)
    x[3] = 0
    codes, scales, exps = oa.rows(x, fmt)
    assert codes.shape == (20, 64) and scales.shape == (20, 128 // ms.BLOCK[fmt])
    assert np.array_equal(oa.row_values(codes, scales, exps, fmt, 72), ms.values(*ms.quantize(x, fmt), fmt, 72))
    if fmt == "mxfp4":
        assert np.array_equal(exps, scales.max(1).astype(int) - 127) and exps[3] == -127


# ---- refusals of the C entry points ----

P = [i << 44 for i in range(1, 12)]


class Cache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), *[(n, ctypes.c_int64) for n in ("pages", "page_size", "heads", "head_dim")],
                *[(n, ctypes.c_void_p) for n in ("codes", "scales", "exponents")]]


class Batch(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("batch", ctypes.c_int64), *[(n, ctypes.c_void_p) for n in ("starts", "lengths", "page_table")],
                ("table_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64)]


class Turn(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("pairs", ctypes.c_int64), ("scale", ctypes.c_double), ("interleaved", ctypes.c_int)]


def cache(**k):
    return Cache(**{**dict(format=0, pages=10, page_size=16, heads=2, head_dim=64, codes=P[0], scales=P[1], exponents=P[2]), **k})


def batch(**k):
    return Batch(**{**dict(tokens=4, batch=2, starts=P[3], lengths=P[4], page_table=P[5], table_pages=3, table_stride=3), **k})


def turn(**k):
    return Turn(**{**dict(turns=P[6], pairs=32, scale=1.0, interleaved=0), **k})


BAD_CACHES = [(dict(format=2), 1), (dict(pages=-1), 1), (dict(page_size=8), 1), (dict(page_size=48), 1), (dict(page_size=1 << 17), 1),
              (dict(heads=0), 1), (dict(heads=4097), 2), (dict(head_dim=0), 1), (dict(head_dim=257), 2), (dict(pages=1 << 40), 2),
              (dict(codes=None), 1), (dict(scales=None), 1), (dict(exponents=None), 1), (dict(codes=P[0] + 8), 1), (dict(scales=P[1] + 4), 1),
              (dict(exponents=P[2] + 1), 1)]
BAD_BATCHES = [(dict(tokens=-1), 1), (dict(batch=-1), 1), (dict(table_pages=-1), 1), (dict(tokens=(1 << 28) + 1), 2), (dict(batch=1 << 29), 2),
               (dict(starts=None), 1), (dict(lengths=None), 1), (dict(page_table=None), 1), (dict(starts=P[3] + 2), 1), (dict(lengths=P[4] + 1), 1),
               (dict(page_table=P[5] + 2), 1), (dict(table_stride=2), 1)]
BAD_STRIDES = [(127, 64), (128, 63), (-128, 64), (1 << 62, 64), (64, 64)]  # of 4 tokens and 2 heads of 64


def test_cache_layout(lib):
    w, n = ctypes.c_int64(), ctypes.c_int64()
    for dim, width in ((1, 64), (64, 64), (65, 128), (128, 128), (129, 256), (256, 256)):
        assert lib.dd_mx4_cache_layout(0, dim, ctypes.byref(w), ctypes.byref(n)) == 0 and (w.value, n.value) == (width, width // 32)
        assert ddg.mx4_cache_layout(dim, "nvfp4") == (width, width // 16)
    assert lib.dd_mx4_cache_layout(0, 257, None, None) == 2 and lib.dd_mx4_cache_layout(0, 0, None, None) == 1
    assert lib.dd_mx4_cache_layout(7, 64, None, None) == 1


def test_append_refusals(lib):
    def call(c=cache(), b=batch(), type=1, k=P[7], kt=128, kh=64, v=P[8], vt=128, vh=64, r=None):
        return lib.dd_mx4_cache_append(ctypes.byref(c) if c else None, ctypes.byref(b) if b else None, type, k, kt, kh, v, vt, vh,
                                       ctypes.byref(r) if r else None, None)

    for k, status in BAD_CACHES:
        assert call(c=cache(**k)) == status, k
    for k, status in BAD_BATCHES:
        assert call(b=batch(**k)) == status, k
    for t, h in BAD_STRIDES:
        assert call(kt=t, kh=h) == 1 and call(vt=t, vh=h) == 1, (t, h)
    assert call(c=None) == 1 and call(b=None) == 1 and call(type=3) == 1
    assert call(k=None) == 1 and call(v=P[8] + 1) == 1 and call(type=0, k=P[7] + 2) == 1
    assert call(k=P[0]) == 1 and call(v=P[1]) == 1 and call(k=P[2] + 16) == 1          # in the cache
    assert call(b=batch(page_table=P[0] + 64)) == 1 and call(b=batch(starts=P[2])) == 1
    for r in (turn(pairs=-1), turn(pairs=33), turn(turns=None), turn(turns=P[6] + 4), turn(interleaved=2), turn(turns=P[0])):
        assert call(r=r) == 1
    assert call(b=batch(tokens=0)) == 0 and call(b=batch(batch=0)) == 0


def test_read_refusals(lib):
    def call(c=cache(), b=batch(), type=1, k=P[7], kt=128, kh=64, v=P[8], vt=128, vh=64):
        return lib.dd_mx4_cache_read(ctypes.byref(c) if c else None, ctypes.byref(b) if b else None, type, k, kt, kh, v, vt, vh, None)

    for k, status in BAD_CACHES:
        assert call(c=cache(**k)) == status, k
    for k, status in BAD_BATCHES:
        assert call(b=batch(**k)) == status, k
    for t, h in BAD_STRIDES:
        assert call(kt=t, kh=h) == 1 and call(vt=t, vh=h) == 1, (t, h)
    assert call(c=None) == 1 and call(b=None) == 1 and call(type=-1) == 1
    assert call(k=None) == 1 and call(v=P[7]) == 1 and call(v=P[7] + 200) == 1          # over one another
    assert call(kt=256, vt=256, v=P[7] + 254) == 1 and call(kt=255, vt=255, v=P[7] + 256) == 1
    assert call(k=P[1]) == 1 and call(v=P[4]) == 1 and call(v=P[5]) == 1 and call(k=P[3]) == 1
    assert call(b=batch(tokens=0)) == 0


def test_attention_refusals(lib):
    def call(c=cache(), b=batch(), type=1, heads=4, q=P[7], qt=256, qh=64, window=0, sinks=0, out=P[8], ot=256, oh=64):
        return lib.dd_mx4_attention(ctypes.byref(c) if c else None, ctypes.byref(b) if b else None, type, heads, q, qt, qh, window, sinks, 1.0,
                                    out, ot, oh, None)

    for k, status in BAD_CACHES:
        assert call(c=cache(**k)) == status, k
    for k, status in BAD_BATCHES:
        assert call(b=batch(**k)) == status, k
    for t, h in BAD_STRIDES:
        assert call(qt=t, qh=h) == 1 and call(ot=t, oh=h) == 1, (t, h)
    assert call(c=None) == 1 and call(b=None) == 1 and call(type=0) == 1                # 16-bit queries only
    assert call(heads=3) == 1 and call(heads=0) == 1 and call(heads=4098) == 2
    assert call(window=-1) == 1 and call(sinks=-1) == 1
    assert call(q=None) == 1 and call(out=None) == 1 and call(out=P[7]) == 1 and call(out=P[7] + 512) == 1
    assert call(out=P[0]) == 1 and call(out=P[3]) == 1 and call(out=P[5]) == 1
    assert call(b=batch(tokens=0)) == 0 and call(b=batch(batch=0)) == 0


def test_rotary_refusals(lib):
    def call(type=1, T=4, H=2, D=64, x=P[0], xt=128, xh=64, p=P[1], wide=1, r=turn(), inverse=0, y=P[2], yt=128, yh=64):
        return lib.dd_rotary(type, T, H, D, x, xt, xh, p, wide, ctypes.byref(r) if r else None, inverse, y, yt, yh, None)

    assert call(type=3) == 1 and call(T=-1) == 1 and call(H=-1) == 1 and call(D=-1) == 1
    assert call(T=(1 << 28) + 1) == 2 and call(H=4097) == 2 and call(D=4097, r=turn()) == 2
    assert call(wide=2) == 1 and call(inverse=2) == 1 and call(r=None) == 1
    for r in (turn(pairs=-1), turn(pairs=33), turn(turns=None), turn(turns=P[6] + 4), turn(interleaved=2)):
        assert call(r=r) == 1
    for t, h in BAD_STRIDES:
        assert call(xt=t, xh=h) == 1 and call(yt=t, yh=h) == 1, (t, h)
    assert call(x=None) == 1 and call(y=None) == 1 and call(p=None) == 1 and call(p=P[1] + 4) == 1 and call(wide=0, p=P[1] + 2) == 1
    assert call(y=P[0] + 128) == 1 and call(y=P[0], yt=256) == 1 and call(y=P[1]) == 1 and call(y=P[6]) == 1
    assert call(T=0) == 0 and call(H=0) == 0


def test_unknown_packed_calls_are_refused(lib):
    for call in (6, 15, 20):
        assert lib.dd_call_packed(call, bytes(400)) == 1
    assert lib.dd_call_packed(19, None) == 1


# ---- refusals of the binding ----

class Stand:
    """What the binding asks of a CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, device=0, stride=None, contiguous=True):
        self.shape, self.dtype, self.index, self.device = tuple(shape), dtype, device, f"cuda:{device}"
        steps = [1]
        for n in reversed(self.shape[1:]):
            steps.insert(0, steps[0] * n)
        self.steps, self.contiguous = tuple(stride or steps), contiguous

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.steps if i is None else self.steps[i]

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 40

    def is_contiguous(self):
        return self.contiguous

    def element_size(self):
        return self.dtype.itemsize

    def is_floating_point(self):
        return self.dtype.is_floating_point

    def is_complex(self):
        return False

    def numel(self):
        return int(np.prod(self.shape))


@pytest.fixture
def binding(monkeypatch):
    torch = pytest.importorskip("torch")
    lp._torch()
    calls = []
    monkeypatch.setattr(lp, "_Tensor", Stand)
    monkeypatch.setattr(lp, "_empty", lambda shape, dtype, device: Stand(shape, dtype))
    monkeypatch.setattr(lp, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(lp, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(lp, "_call", lambda name, *args: calls.append((name, args, lp._PACKED[name][1](*args))))
    return torch, calls


def parts(torch, fmt="mxfp4", dim=64, heads=2, page=16, device=0):
    width, scales = ddg.mx4_cache_layout(dim, fmt)
    shape = (5, 2, heads, page)
    held = ddg.MX4Cache(Stand((*shape, width // 2), torch.uint8, device), Stand((*shape, scales), torch.uint8, device), Stand(shape, torch.int8, device), dim, fmt)
    plan = [Stand((3,), torch.int32, device), Stand((2,), torch.int32, device), Stand((2, 4), torch.int32, device)]
    return held, plan


def every_call(torch, device=0):
    held, plan = parts(torch, device=device)
    half = lambda h: Stand((6, h, 64), torch.bfloat16, device)  # noqa: E731
    table = ddg.Rotary(Stand((16,), torch.int64, device))
    p = Stand((6,), torch.int64, device)
    return {
        "dd_rotary": [lambda: ddg.rotary(half(3), p, table), lambda: ddg.rotary_backward(half(3), p, table)],
        "dd_mx4_cache_append": [lambda: ddg.mx4_cache_append(held, half(2), half(2), *plan), lambda: ddg.mx4_cache_append(held, half(2), half(2), *plan, rotary=table)],
        "dd_mx4_cache_read": [lambda: ddg.mx4_cache_read(held, 6, *plan)],
        "dd_mx4_attention": [lambda: ddg.mx4_attention(half(8), held, *plan, window=9, sinks=2)],
    }


def test_sound_calls_reach_the_library(binding):
    torch, calls = binding
    for name, runs in every_call(torch).items():
        for run in runs:
            run()
            assert calls.pop()[0] == name and not calls


def test_tensors_of_another_device_than_the_current_one_are_refused(binding, monkeypatch):
    torch, calls = binding
    monkeypatch.setattr(lp, "_current_device", lambda: 1)
    for runs in every_call(torch).values():
        for run in runs:
            with pytest.raises(ValueError, match="current"):
                run()
    assert not calls


def test_rotary_arguments(binding):
    torch, calls = binding
    x, p, table = Stand((6, 3, 64), torch.float16), Stand((6,), torch.int32), ddg.Rotary(Stand((16,), torch.int64))
    bad = [((Stand((6, 64), torch.float16), p, table), {}, TypeError), ((Stand((6, 3, 64), torch.int32), p, table), {}, TypeError),
           ((Stand((6, 3, 64), torch.float16, stride=(192, 1, 3)), p, table), {}, ValueError),
           ((x, Stand((5,), torch.int32), table), {}, ValueError), ((x, Stand((6,), torch.float32), table), {}, TypeError),
           ((x, Stand((6,), torch.int16), table), {}, TypeError), ((x, Stand((6,), torch.int32, contiguous=False), table), {}, ValueError),
           ((x, Stand((6,), torch.int32, 1), table), {}, ValueError), ((x, p, ddg.Rotary(Stand((33,), torch.int64))), {}, ValueError),
           ((x, p, ddg.Rotary(Stand((16,), torch.float64))), {}, TypeError), ((x, p, ddg.Rotary(Stand((4, 4), torch.int64))), {}, TypeError),
           ((x, p, ddg.Rotary(Stand((16,), torch.int64, 1))), {}, ValueError),
           ((x, p, table), dict(out=Stand((6, 3, 64), torch.bfloat16)), TypeError), ((x, p, table), dict(out=Stand((6, 2, 64), torch.float16)), ValueError),
           ((x, p, table), dict(out=Stand((6, 3, 64), torch.float16, 1)), ValueError)]
    for args, more, error in bad:
        for call in (ddg.rotary, ddg.rotary_backward):
            with pytest.raises(error):
                call(*args, **more)
    assert not calls
    for wrong in (dict(dim=7), dict(dim=-2), dict(dim=8, scaling="cubic"), dict(dim=2, scaling="base", factor=2.0), dict(dim=8, factor=0.0),
                  dict(dim=8, frequencies=[1.0]), dict(dim=8, scaling="bands", bands=(4.0, 4.0)), dict(dim=4, frequencies=[1.0, float("inf")])):
        with pytest.raises(ValueError):
            ddg.rotary_table(**wrong, device="cpu")


def test_cache_and_batch_arguments(binding):
    torch, calls = binding
    held, plan = parts(torch)
    half = lambda *s, d=0: Stand(s, torch.bfloat16, d)  # noqa: E731

    def each(held, plan):
        return [lambda: ddg.mx4_cache_append(held, half(6, 2, 64), half(6, 2, 64), *plan), lambda: ddg.mx4_cache_read(held, 6, *plan),
                lambda: ddg.mx4_attention(half(6, 4, 64), held, *plan)]

    def swapped(**k):
        return ddg.MX4Cache(**{**dict(codes=held.codes, scales=held.scales, exponents=held.exponents, head_dim=64, fmt="mxfp4"), **k})

    shape = (5, 2, 2, 16)
    for wrong in (swapped(fmt="int4"), swapped(head_dim=0), swapped(head_dim=300), swapped(head_dim=128), swapped(fmt="nvfp4"), swapped(codes=None),
                  swapped(codes=Stand((*shape, 32), torch.float32)), swapped(codes=Stand((*shape, 32), torch.uint8, contiguous=False)),
                  swapped(codes=Stand((5, 3, 2, 16, 32), torch.uint8)), swapped(scales=Stand((*shape, 3), torch.uint8)), swapped(scales=Stand((*shape, 2), torch.uint8, 1)),
                  swapped(exponents=Stand((*shape, 1), torch.int8)), swapped(exponents=Stand(shape, torch.int32))):
        for call in each(wrong, plan):
            with pytest.raises((ValueError, TypeError)):
                call()
    starts, lengths, table = plan
    for wrong in ([Stand((3,), torch.int64), lengths, table], [Stand((2,), torch.int32), lengths, table], [starts, Stand((3,), torch.int32), table],
                  [starts, lengths, Stand((2, 2, 2), torch.int32)], [starts, lengths, Stand((2, 4), torch.int32, stride=(1, 2))], [starts, lengths, None],
                  [Stand((3,), torch.int32, 1), lengths, table], [Stand((3,), torch.int32, contiguous=False), lengths, table]):
        for call in each(held, wrong):
            with pytest.raises((ValueError, TypeError)):
                call()
    for wrong in (lambda: ddg.mx4_cache_append(held, half(6, 3, 64), half(6, 3, 64), *plan), lambda: ddg.mx4_cache_append(held, half(6, 2, 64), half(5, 2, 64), *plan),
                  lambda: ddg.mx4_cache_append(held, half(6, 2, 64), Stand((6, 2, 64), torch.float16), *plan),
                  lambda: ddg.mx4_cache_append(held, half(6, 2, 64, d=1), half(6, 2, 64, d=1), *plan),
                  lambda: ddg.mx4_cache_append(held, half(6, 2, 64), half(6, 2, 64), *plan, rotary=ddg.Rotary(Stand((33,), torch.int64))),
                  lambda: ddg.mx4_cache_read(held, 6, *plan, dtype=torch.int8), lambda: ddg.mx4_cache_read(held, 6, *plan, out=(half(5, 2, 64), half(6, 2, 64))),
                  lambda: ddg.mx4_attention(half(6, 3, 64), held, *plan), lambda: ddg.mx4_attention(half(6, 4, 32), held, *plan),
                  lambda: ddg.mx4_attention(Stand((6, 4, 64), torch.float32), held, *plan), lambda: ddg.mx4_attention(half(6, 0, 64), held, *plan),
                  lambda: ddg.mx4_attention(half(6, 4, 64), held, *plan, window=-1), lambda: ddg.mx4_attention(half(6, 4, 64), held, *plan, sinks=-2),
                  lambda: ddg.mx4_attention(half(6, 4, 64), held, *plan, out=half(6, 2, 64))):
        with pytest.raises((ValueError, TypeError)):
            wrong()
    assert not calls


@pytest.mark.parametrize("scale", (float("nan"), float("inf"), -float("inf"), 3e38))
def test_attention_refuses_scales_that_are_not_finite(lib, scale):
    """In base 2, too: 3e38 log2(e) is none."""
    for tokens, window in ((4, 0), (400, 3)):
        assert lib.dd_mx4_attention(ctypes.byref(cache()), ctypes.byref(batch(tokens=tokens)), 1, 4, P[7], 256, 64, window, 0, scale, P[9], 256, 64, None) == 1
