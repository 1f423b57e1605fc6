"""Calls of the 4-bit and feed-forward entry points that must not reach the GPU
(no GPU needed)."""
import ctypes
import pathlib
import re

import pytest

import extended_precision_gemm_gb300 as ddg
from extended_precision_gemm_gb300 import low_precision as lp


@pytest.fixture(scope="module")
def lib():
    return ddg.load()


# ---- tensors of a device that is not the current one ----

class Stand:
    """What the binding asks of a contiguous CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, device=0):
        self.shape = (shape,) if isinstance(shape, int) else tuple(shape)
        self.dtype, self.device = dtype, device

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = (self.shape[1], 1) if len(self.shape) == 2 else (1,)
        return s if i is None else s[i]

    def numel(self):
        n = 1
        for v in self.shape:
            n *= v
        return n

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 1 << 40

    def is_contiguous(self):
        return True


@pytest.fixture
def binding(monkeypatch):
    """The binding with stand-ins for tensors, the stream and the library; the calls that reach the library."""
    pytest.importorskip("torch")
    lp._torch()
    calls = []
    monkeypatch.setattr(lp, "_Tensor", Stand)
    monkeypatch.setattr(lp, "_empty", lambda shape, dtype, device: Stand(shape, dtype, device))
    monkeypatch.setattr(lp, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(lp, "_call", lambda name, *args: calls.append(name))
    return calls


def every_call():
    import torch
    half = lambda r, c: Stand((r, c), torch.bfloat16)  # noqa: E731
    q = lambda rows, k: ddg.MX4(Stand((rows, -(-k // 32) * 16), torch.uint8), Stand(lp._scale_bytes(1, rows, k), torch.uint8),  # noqa: E731
                                Stand(rows, torch.int32), rows, k, "nvfp4")
    T, D, F = 5, 64, 96
    x, wg, wu, wd = half(T, D), half(F, D), half(F, D), half(D, F)
    saved = Stand(ddg.ff_gated_saved_size(T, F, torch.bfloat16), torch.uint8)
    return {
        "dd_mx4_quantize": lambda: ddg.mx4_quantize(x, "nvfp4"),
        "dd_mx4_dequantize": lambda: ddg.mx4_dequantize(q(T, D)),
        "dd_mx4_gemm": lambda: ddg.mx4_gemm(q(T, D), q(F, D)),
        "dd_mx4_ff_gated": lambda: ddg.mx4_ff_gated(x, q(2 * F, D), q(D, F)),
        "dd_ff_gated": lambda: ddg.ff_gated(x, wg, wu, wd, save=True),
        "dd_ff_gated_backward": lambda: ddg.ff_gated_backward(x, x, wg, wu, wd, saved),
    }


def test_tensors_of_another_device_than_the_current_one_are_refused(binding, monkeypatch):
    """Launches, workspaces and the default stream are the current device's."""
    monkeypatch.setattr(lp, "_current_device", lambda: 1, raising=False)
    for name, call in every_call().items():
        with pytest.raises(ValueError, match="current"):
            call()
        assert not binding, name


def test_tensors_of_the_current_device_are_taken(binding, monkeypatch):
    monkeypatch.setattr(lp, "_current_device", lambda: 0, raising=False)
    for name, call in every_call().items():
        call()
        assert binding.pop() == name and not binding


# ---- row exponents that are not aligned ----

def test_misaligned_row_exponents_are_refused(lib):
    a, b, c, d, e, f, y = (ctypes.c_void_p(i << 40) for i in range(1, 8))
    for off in (1, 2, 3):
        odd = ctypes.c_void_p((9 << 40) + off)
        assert lib.dd_mx4_quantize(1, 1, 0, 8, 64, a, 64, b, 32, c, odd, None) == 1
        assert lib.dd_mx4_quantize(1, 1, 1, 8, 64, a, 8, b, 32, c, odd, None) == 1
        assert lib.dd_mx4_dequantize(1, 1, 8, 64, a, 32, b, odd, c, 64, None) == 1
        assert lib.dd_mx4_gemm(1, 8, 8, 64, a, 32, b, odd, c, 32, d, e, 1.0, 1, y, 8, None) == 1
        assert lib.dd_mx4_gemm(1, 8, 8, 64, a, 32, b, e, c, 32, d, odd, 1.0, 1, y, 8, None) == 1
        for first, second in ((odd, y), (y, odd)):
            assert lib.dd_mx4_ff_gated(1, 1, 0, 3, 64, 40, a, 64, b, 32, c, first, d, 32, e, second, f, 64, None) == 1
        # without anything to read or write they are not looked at
        assert lib.dd_mx4_quantize(1, 1, 0, 0, 64, a, 64, b, 32, c, odd, None) == 0


# ---- shared memory read in words wider than its elements ----

WIDE = {"uint4": 16, "int4": 16, "float4": 16, "uint2": 8, "int2": 8, "float2": 8, "double2": 16, "ulonglong2": 16}
BYTES = {"uint8_t": 1, "uint16_t": 2, "uint32_t": 4, "int": 4, "float": 4, "uint64_t": 8, "double": 8, **WIDE}


def test_shared_arrays_are_aligned_to_what_is_read_from_them():
    """A __shared__ array that is cast to a wider type says so where it is declared: the compiler places it by its
    elements otherwise, and an unaligned wide access faults."""
    seen = 0
    for path in sorted((pathlib.Path(lp.__file__).parent / "csrc").glob("*.cu*")):
        text = path.read_text()
        for m in re.finditer(r"__shared__\s+(__align__\((\d+)\)\s+)?(\w+)\s+(\w+)((?:\[[^;]*?\])+);", text):
            align, elem, name = int(m.group(2) or 0), m.group(3), m.group(4)
            end = re.search(r"\n}", text[m.end():])
            body = text[m.end(): m.end() + (end.start() if end else 0)]
            for cast in re.finditer(r"reinterpret_cast<(?:const )?(?:volatile )?(\w+)\s*\*>\(&?" + name + r"\b", body):
                need = BYTES.get(cast.group(1), 1)
                seen += 1
                assert max(align, BYTES.get(elem, 1)) >= need, f"{path.name}: {name} is read as {cast.group(1)}"
    assert seen > 0
