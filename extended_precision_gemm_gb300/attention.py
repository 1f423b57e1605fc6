"""The attention side of a layer around a cache in 4 bits: rotary positions, a
paged key/value cache in the 4-bit microscaled formats, and attention over it:
argument marshalling for the entry points of ``ddgemm.h`` (layouts, formulas and
roundings are defined there).

    table = rotary_table(128, base=500000.0)
    q = rotary(q, positions, table)                       # tokens x heads x dim
    dx = rotary_backward(dy, positions, table)
    cache = mx4_cache(pages, page_size, heads, 128, "mxfp4")
    mx4_cache_append(cache, k, v, starts, lengths, page_table, rotary=table)
    y = mx4_attention(q, cache, starts, lengths, page_table)
    k, v = mx4_cache_read(cache, tokens, starts, lengths, page_table)

A batch of sequences is (starts, lengths, page_table), int32 on the device: the
call's tokens starts[b] .. starts[b + 1] are the last ones of sequence b, which has
lengths[b] tokens in the cache (after the append) in the pages page_table[b].
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import struct

import extended_precision_gemm_gb300 as _ddg

from . import low_precision as _lp
from .low_precision import MX4_FORMATS, _lookup, _type

_lp._PACKED.update({
    "dd_rotary": (16, struct.Struct("=11qd6q").pack),
    "dd_mx4_cache_append": (17, struct.Struct("=24qd2q").pack),
    "dd_mx4_cache_read": (18, struct.Struct("=23q").pack),
    "dd_mx4_attention": (19, struct.Struct("=22qd4q").pack),
})


def _heads(t, name, dtype=None):
    """(tokens, heads, dim, strides of tokens and heads) of a 3-D CUDA tensor whose
    last dimension is contiguous (of `dtype`)."""
    if _lp._types is None:
        _lp._torch()
    if not isinstance(t, _lp._Tensor) or t.dim() != 3 or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be a 3-D {dtype or 'torch'} tensor (tokens, heads, dim)")
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    T, H, D = t.shape
    st, sh, unit = t.stride()
    if D > 1 and unit != 1 and T > 0 and H > 0:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return T, H, D, st, sh


def _result(out, shape, dtype, like, name, stream):
    """(`out` checked, or a new tensor on like's device, its strides); a new one is
    recorded on `stream`, which may not be the one it was allocated for."""
    if out is None:
        out = _lp._empty(shape, dtype=dtype, device=like.device)
        if stream is not None:
            out.record_stream(stream)
        return out, shape[1] * shape[2], shape[2]
    T, H, D, st, sh = _heads(out, name, dtype)
    if (T, H, D) != tuple(shape) or out.get_device() != like.get_device():
        raise ValueError(f"{name} must be {tuple(shape)} on {like.device}")
    return out, st, sh


def _here(device, *tensors):
    for t in tensors:
        if t.get_device() != device:
            raise ValueError("tensors must be on the same device")


# ---- rotary positions ----

@dataclasses.dataclass
class Rotary:
    """A rotation by positions: pair i turns by turns[i] / 2^64 turns a position
    (int64 or uint64, on the device) and is multiplied by scale; its elements are i
    and len(turns) + i, or with `interleaved` 2 i and 2 i + 1."""

    turns: object
    scale: float = 1.0
    interleaved: bool = False

    def _words(self, device):
        if _lp._types is None:
            _lp._torch()
        t = self.turns
        if not isinstance(t, _lp._Tensor) or t.dim() != 1 or t.element_size() != 8 or t.is_floating_point() or t.is_complex():
            raise TypeError("turns must be a 1-D int64 or uint64 CUDA tensor")
        if not t.is_contiguous():
            raise ValueError("turns must be contiguous")
        _here(device, t)
        n = t.shape[0]
        return t.data_ptr() if n else 0, n, float(self.scale), 1 if self.interleaved else 0


ROTARY_SCALINGS = ("linear", "base", "bands")


def rotary_table(dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str | None = None, factor: float = 1.0,
                 original: int = 4096, bands=(1.0, 32.0), frequencies=None, scale: float | None = None, device=None) -> Rotary:
    """The rotation of the first `dim` elements of a head: pair i turns by
    base^(-2 i / dim) radians a position, or by frequencies[i].  For contexts `factor`
    times as long as the `original` one:

      "linear"  every frequency over factor;
      "base"    the base times factor^(dim / (dim - 2));
      "bands"   pairs that turn bands[1] times or more over the original context
                stay, those that turn bands[0] times or fewer are divided by factor,
                those between by a mixture, and scale is 0.1 ln(factor) + 1."""
    torch = _lp._torch()
    if dim < 0 or dim % 2:
        raise ValueError("dim must be even")
    if scaling is not None and scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(ROTARY_SCALINGS)}")
    if not (factor > 0 and math.isfinite(factor)):
        raise ValueError("factor must be positive")
    if scaling == "base":
        if dim <= 2:
            raise ValueError("scaling by the base needs a dim above 2")
        base = base * factor ** (dim / (dim - 2))
    if frequencies is None:
        f = [base ** (-i / dim) for i in range(0, dim, 2)]
    else:
        f = [float(x) for x in frequencies]
        if len(f) != dim // 2:
            raise ValueError("frequencies must be dim / 2 numbers")
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "bands":
        low, high = bands
        if not low < high:
            raise ValueError("bands must be two numbers, the lower one first")
        keep = [min(1.0, max(0.0, (x * original / (2 * math.pi) - low) / (high - low))) for x in f]
        f = [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]
        if scale is None:
            scale = 0.1 * math.log(factor) + 1.0
    if not all(math.isfinite(x) for x in f):
        raise ValueError("frequencies must be finite")
    turns = [int(x / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for x in f]
    turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device or torch.device("cuda"))
    return Rotary(turns, 1.0 if scale is None else float(scale), interleaved)


def _rotate(x, name, positions, table, inverse, out, stream):
    T, H, D, st, sh = _heads(x, name)
    code = _type(x.dtype, name)
    device = x.get_device()
    if not isinstance(positions, _lp._Tensor) or positions.dim() != 1 or positions.element_size() not in (4, 8) \
            or positions.is_floating_point() or positions.is_complex() or (positions.element_size() == 4 and positions.dtype is not _lp._int32):
        raise TypeError("positions must be a 1-D int32 or int64 CUDA tensor")
    if positions.shape[0] != T or not positions.is_contiguous():
        raise ValueError("positions must be contiguous, one for each token")
    _here(device, positions)
    words = table._words(device)
    if 2 * words[1] > D:
        raise ValueError("the rotation is wider than a head")
    y, yt, yh = _result(out, (T, H, D), x.dtype, x, "out", stream)
    _lp._call("dd_rotary", code, T, H, D, x.data_ptr(), st, sh, positions.data_ptr(), 1 if positions.element_size() == 8 else 0,
          *words, inverse, y.data_ptr(), yt, yh, _lp._stream(stream, x))
    return y


def rotary(x, positions, table: Rotary, out=None, stream=None):
    """x (tokens, heads, dim; float32, bfloat16 or float16, any strides of tokens and
    heads) turned at `positions` (int32 or int64); out may be x."""
    return _rotate(x, "x", positions, table, 0, out, stream)


def rotary_backward(dy, positions, table: Rotary, out=None, stream=None):
    """dx from dy: the transposed rotation; out may be dy."""
    return _rotate(dy, "dy", positions, table, 1, out, stream)


# ---- the cache ----

@dataclasses.dataclass
class MX4Cache:
    """A paged key/value cache in 4-bit microscaled form (layout: ddgemm.h).

    codes: uint8 (pages, 2, heads, page_size, width / 2); scales: uint8 (pages, 2,
    heads, page_size, width / 32 or width / 16); exponents: int8 (pages, 2, heads,
    page_size); keys are 0 and values 1, width is head_dim filled up to 64, 128 or 256.
    """

    codes: object
    scales: object
    exponents: object
    head_dim: int
    fmt: str

    @property
    def pages(self):
        return self.codes.shape[0]

    @property
    def heads(self):
        return self.codes.shape[2]

    @property
    def page_size(self):
        return self.codes.shape[3]

    def _words(self):
        """(device, the members of ddgemm_mx4_cache), checked; the one test that a
        sound cache passes comes first, the reasons after."""
        if _lp._types is None:
            _lp._torch()
        c, s, e, dim = self.codes, self.scales, self.exponents, self.head_dim
        fmt = MX4_FORMATS.get(self.fmt)
        if fmt is not None and isinstance(c, _lp._Tensor) and isinstance(s, _lp._Tensor) and isinstance(e, _lp._Tensor) and 1 <= dim <= 256:
            shape, device = c.shape, c.get_device()
            width = 64 if dim <= 64 else 128 if dim <= 128 else 256
            if (len(shape) == 5 and c.dtype is _lp._uint8 and s.dtype is _lp._uint8 and e.element_size() == 1 and device >= 0
                    and s.get_device() == device and e.get_device() == device and shape[1] == 2 and shape[4] == width // 2
                    and s.shape == (*shape[:4], width // (16 if fmt else 32)) and e.shape == shape[:4]
                    and c.is_contiguous() and s.is_contiguous() and e.is_contiguous()):
                return device, (fmt, shape[0], shape[3], shape[2], dim, c.data_ptr(), s.data_ptr(), e.data_ptr())
        self._refuse()

    def _refuse(self):
        """Raises for what _words found wrong."""
        fmt = _lookup(MX4_FORMATS, self.fmt, "fmt")
        parts = {"codes": self.codes, "scales": self.scales, "exponents": self.exponents}
        for name, t in parts.items():
            if not isinstance(t, _lp._Tensor) or t.element_size() != 1 or t.is_floating_point() or not t.is_cuda:
                raise TypeError(f"cache.{name} must be a CUDA tensor of bytes")
        if not 1 <= self.head_dim <= 256:
            raise ValueError("cache.head_dim must be 1 to 256")
        width = 64 if self.head_dim <= 64 else 128 if self.head_dim <= 128 else 256
        if self.codes.dim() != 5 or self.codes.shape[1] != 2 or self.codes.shape[4] != width // 2:
            raise ValueError(f"cache.codes must be (pages, 2, heads, page_size, {width // 2})")
        shape = tuple(self.codes.shape[:4])
        if tuple(self.scales.shape) != (*shape, width // (16 if fmt else 32)) or tuple(self.exponents.shape) != shape:
            raise ValueError(f"cache.scales must be {(*shape, width // (16 if fmt else 32))} and cache.exponents {shape}")
        if not all(t.is_contiguous() for t in parts.values()):
            raise ValueError("the tensors of the cache must be contiguous")
        raise ValueError("the tensors of the cache must be on the same device, codes and scales uint8")


def mx4_cache_layout(head_dim: int, fmt: str = "mxfp4"):
    """(width, bytes of scales) of a row."""
    width, scales = ctypes.c_int64(), ctypes.c_int64()
    _ddg._check("dd_mx4_cache_layout", _ddg.load().dd_mx4_cache_layout(_lookup(MX4_FORMATS, fmt, "fmt"), head_dim,
                                                                      ctypes.byref(width), ctypes.byref(scales)))
    return width.value, scales.value


def mx4_cache(pages: int, page_size: int, heads: int, head_dim: int, fmt: str = "mxfp4", device=None) -> MX4Cache:
    """An empty cache of pages * page_size tokens (page_size a power of two from 16 to
    65536) of `heads` key and value heads."""
    torch = _lp._torch()
    width, scales = mx4_cache_layout(head_dim, fmt)
    device = device or torch.device("cuda")
    shape = (pages, 2, heads, page_size)
    return MX4Cache(torch.zeros((*shape, width // 2), dtype=torch.uint8, device=device),
                    torch.zeros((*shape, scales), dtype=torch.uint8, device=device),
                    torch.zeros(shape, dtype=torch.int8, device=device), head_dim, fmt)


def _batch(device, tokens, starts, lengths, page_table):
    """The members of ddgemm_batch, checked."""
    for name, t, dims in (("starts", starts, 1), ("lengths", lengths, 1), ("page_table", page_table, 2)):
        if not isinstance(t, _lp._Tensor) or t.dtype is not _lp._int32 or t.dim() != dims:
            raise TypeError(f"{name} must be a {dims}-D int32 CUDA tensor")
        if t.get_device() != device:
            raise ValueError("tensors must be on the same device")
    batch, n = page_table.shape
    if lengths.shape[0] != batch or starts.shape[0] != batch + 1:
        raise ValueError("starts, lengths and page_table must be of batch + 1, batch and batch sequences")
    ld, unit = page_table.stride()
    if not starts.is_contiguous() or not lengths.is_contiguous() or (n > 1 and unit != 1 and batch > 0):
        raise ValueError("starts, lengths and the rows of page_table must be contiguous")
    return tokens, batch, starts.data_ptr(), lengths.data_ptr(), page_table.data_ptr(), n, ld if batch > 1 else n


def mx4_cache_append(cache: MX4Cache, k, v, starts, lengths, page_table, rotary: Rotary | None = None, stream=None) -> MX4Cache:
    """Quantises the batch's tokens k and v (tokens, heads, head_dim; float32, bfloat16
    or float16) into the cache; with `rotary` keys are turned at their positions on
    the way.  Returns the cache."""
    device, words = cache._words()
    T, H, D, kt, kh = _heads(k, "k")
    code = _type(k.dtype, "k")
    shape = _heads(v, "v", k.dtype)
    if (T, H, D) != shape[:3] or H != cache.heads or D != cache.head_dim:
        raise ValueError(f"k and v must be (tokens, {cache.heads}, {cache.head_dim})")
    _here(device, k, v)
    turn = (0, 0, 1.0, 0) if rotary is None else rotary._words(device)
    if 2 * turn[1] > D:
        raise ValueError("the rotation is wider than a head")
    _lp._call("dd_mx4_cache_append", *words, *_batch(device, T, starts, lengths, page_table), code, k.data_ptr(), kt, kh,
          v.data_ptr(), *shape[3:], *turn, _lp._stream(stream, k))
    return cache


def mx4_cache_read(cache: MX4Cache, tokens: int, starts, lengths, page_table, dtype=None, out=None, stream=None):
    """(k, v) that the cache has for the batch's tokens, each (tokens, heads,
    head_dim), bfloat16 by default, which holds them exactly.  Rows of no sequence
    are left as they are (and are not set in new tensors)."""
    device, words = cache._words()
    k, v = out if out is not None else (None, None)
    dtype = dtype or (k.dtype if k is not None else _lp._torch().bfloat16)
    code = _type(dtype, "dtype")
    shape = (tokens, cache.heads, cache.head_dim)
    k, kt, kh = _result(k, shape, dtype, cache.codes, "out", stream)
    v, vt, vh = _result(v, shape, dtype, cache.codes, "out", stream)
    _lp._call("dd_mx4_cache_read", *words, *_batch(device, tokens, starts, lengths, page_table), code, k.data_ptr(), kt, kh,
          v.data_ptr(), vt, vh, _lp._stream(stream, k))
    return k, v


def mx4_attention(q, cache: MX4Cache, starts, lengths, page_table, window: int = 0, sinks: int = 0, scale: float | None = None,
                  out=None, stream=None):
    """softmax(scale q k^T) v for the batch's tokens over the cache (scale: 1 /
    sqrt(head_dim) by default): q (tokens, query heads, head_dim; bfloat16 or float16),
    query heads a multiple of the cache's.  A token sees those of its sequence up to
    itself; with a window the last `window` of them and the first `sinks`.  Rows of no
    sequence are left as they are (and are not set in a new tensor)."""
    device, words = cache._words()
    T, H, D, qt, qh = _heads(q, "q")
    code = _type(q.dtype, "q", sixteen=True)
    heads = words[3]
    if D != cache.head_dim or heads == 0 or H == 0 or H % heads:
        raise ValueError(f"q must be (tokens, a multiple of {heads}, {cache.head_dim})")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    _here(device, q)
    y, yt, yh = _result(out, (T, H, D), q.dtype, q, "out", stream)
    _lp._call("dd_mx4_attention", *words, *_batch(device, T, starts, lengths, page_table), code, H, q.data_ptr(), qt, qh, window,
          sinks, D ** -0.5 if scale is None else scale, y.data_ptr(), yt, yh, _lp._stream(stream, q))
    return y
