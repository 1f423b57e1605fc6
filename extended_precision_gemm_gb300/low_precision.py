"""4-bit microscaled matrices, their products, and the gated feed-forward
block in 16 and in 4 bits: argument marshalling for the entry points of
``ddgemm.h`` (formats, layouts and roundings are defined there).

    q = mx4_quantize(x, "mxfp4")            # rows; cols=True: columns
    C = mx4_gemm(a, b)                      # a: M x K, b: N x K, C = a b^T
    y, saved = ff_gated(x, Wg, Wu, Wd, save=True)
    dx, dWg, dWu, dWd = ff_gated_backward(dy, x, Wg, Wu, Wd, saved)
    w_in, w_out = mx4_ff_weights(Wg, Wu, Wd, "mxfp4")
    y = mx4_ff_gated(x, w_in, w_out)
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import struct

import extended_precision_gemm_gb300 as _ddg

MX4_FORMATS = {"mxfp4": 0, "nvfp4": 1}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


_types = _types16 = _uint8 = _int32 = _Tensor = _empty = _raw_stream = _current_device = None


def _torch():
    """torch, imported on the first call (with the lookups that every call makes)."""
    global _types, _types16, _uint8, _int32, _Tensor, _empty, _raw_stream, _current_device
    import torch
    if _types is None:
        _uint8, _int32, _Tensor, _empty = torch.uint8, torch.int32, torch.Tensor, torch.empty
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _types16 = {torch.bfloat16: 1, torch.float16: 2}
        _types = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    return torch


def _stream(stream, t):
    """The handle of `stream`, or of the current stream of t's device, which has
    to be the current one: launches and workspaces are on that, and so is the
    default stream, whose handle is the same on every device."""
    if t.get_device() != _current_device():
        raise ValueError("tensors must be on the current CUDA device (torch.cuda.device)")
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _torch().cuda.current_stream(t.device).cuda_stream


# dd_call_packed's number of an entry point, and how its arguments are packed
_PACKED = {
    "dd_mx4_quantize": (0, struct.Struct("=12q").pack),
    "dd_mx4_dequantize": (1, struct.Struct("=11q").pack),
    "dd_mx4_gemm": (2, struct.Struct("=12qd4q").pack),
    "dd_mx4_ff_gated": (3, struct.Struct("=19q").pack),
    "dd_ff_gated": (4, struct.Struct("=18q").pack),
    "dd_ff_gated_backward": (5, struct.Struct("=25q").pack),
}


def _call(name, *args):
    call, pack = _PACKED[name]
    status = (_ddg._lib or _ddg.load()).dd_call_packed(call, pack(*args))
    if status != 0:
        raise _ddg.DDGemmError(name, status)


def _lookup(table, key, name):
    value = table.get(key)
    if value is None:
        raise ValueError(f"{name} must be one of {', '.join(table)}")
    return value


def _type(dtype, name, sixteen=False):
    if _types is None:
        _torch()
    types = _types16 if sixteen else _types
    code = types.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be {' or '.join(str(t) for t in types)}")
    return code


def _matrix(t, name, dtype=None):
    """(rows, columns, leading dimension) of a 2-D CUDA tensor with unit column
    stride (of `dtype`)."""
    if _types is None:
        _torch()
    if not isinstance(t, _Tensor) or t.dim() != 2 or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be a 2-D {dtype or 'torch'} tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    rows, cols = t.shape
    ld, unit = t.stride()
    if cols > 1 and rows > 0 and unit != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if rows <= 1 or cols == 0:
        ld = cols or 1
    elif ld < cols:
        raise ValueError(f"{name} must have rows that do not overlap")
    return rows, cols, ld


def _like(out, shape, dtype, like, name, stream):
    """(`out` checked, or a new tensor on like's device, its leading
    dimension); a new one is recorded on `stream`, which may not be the one it
    was allocated for."""
    if out is None:
        out = _empty(shape, dtype=dtype, device=like.device)
        if stream is not None:
            out.record_stream(stream)
        return out, shape[1] or 1
    rows, cols, ld = _matrix(out, name, dtype)
    if (rows, cols) != tuple(shape) or out.device != like.device:
        raise ValueError(f"{name} must be {tuple(shape)} on {like.device}")
    return out, ld


def _same_device(*tensors):
    index = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != index:
            raise ValueError("tensors must be on the same device")


# ---- 4-bit matrices ----

@dataclasses.dataclass
class MX4:
    """A rows x k matrix in 4-bit microscaled form (layout: ddgemm.h).

    codes: uint8 (rows, k / 2 rounded up to 16) or wider, 16-byte rows; scales:
    uint8, the tiles one after the other; exponents: int32 (rows), nvfp4 only.
    """

    codes: object
    scales: object
    exponents: object
    rows: int
    k: int
    fmt: str

    @property
    def shape(self):
        return (self.rows, self.k)

    def _args(self, name):
        """(device, format, codes, leading dimension, scales, exponents), checked;
        the one test that a sound matrix passes comes first, the reasons after."""
        if _types is None:
            _torch()
        c, s, e, rows, k = self.codes, self.scales, self.exponents, self.rows, self.k
        fmt = MX4_FORMATS.get(self.fmt)
        if fmt is not None and isinstance(c, _Tensor) and isinstance(s, _Tensor):
            shape, stride, device = c.shape, c.stride(), c.get_device()
            width = -(-k // 32) * 16
            if (len(shape) == 2 and c.dtype is _uint8 and s.dtype is _uint8 and device >= 0 and s.get_device() == device
                    and shape[0] == rows and shape[1] >= width and (stride[1] == 1 or rows == 0 or shape[1] <= 1)
                    and s.numel() >= _scale_bytes(fmt, rows, k) and s.is_contiguous()):
                ld = stride[0] if rows > 1 else -(-shape[1] // 16) * 16
                if fmt == 0:
                    return device, 0, c.data_ptr(), ld, s.data_ptr(), 0
                if (isinstance(e, _Tensor) and e.dtype is _int32 and e.get_device() == device and e.numel() >= rows
                        and e.is_contiguous()):
                    return device, 1, c.data_ptr(), ld, s.data_ptr(), e.data_ptr()
        self._refuse(name)

    def _refuse(self, name):
        """Raises for what _args found wrong."""
        fmt = _lookup(MX4_FORMATS, self.fmt, "fmt")
        c, s, e, rows = self.codes, self.scales, self.exponents, self.rows
        width, scale_bytes = _sizes(fmt, rows, self.k)
        if not isinstance(c, _Tensor) or c.dtype != _uint8 or c.dim() != 2 or not c.is_cuda:
            raise TypeError(f"{name}.codes must be a 2-D uint8 CUDA tensor")
        if c.shape[0] != rows or c.shape[1] < width or c.stride(1) != 1:
            raise ValueError(f"{name}.codes must be {rows} rows of at least {width} bytes")
        if not isinstance(s, _Tensor) or s.dtype != _uint8 or not s.is_cuda:
            raise TypeError(f"{name}.scales must be a uint8 CUDA tensor")
        if s.numel() < scale_bytes or not s.is_contiguous():
            raise ValueError(f"{name}.scales must hold {scale_bytes} contiguous bytes")
        if fmt == 1:
            if not isinstance(e, _Tensor) or e.dtype != _int32 or not e.is_cuda:
                raise TypeError(f"{name}.exponents must be an int32 CUDA tensor")
            if e.numel() < rows or not e.is_contiguous():
                raise ValueError(f"{name}.exponents must hold {rows} contiguous values")
        raise ValueError(f"the tensors of {name} must be on the same device")


def _scale_bytes(fmt, rows, k):
    return -(-rows // 128) * -(-k // 256) * (1024 if fmt == 0 else 2048)


def _sizes(fmt, rows, k):
    """dd_mx4_layout for sizes that a tensor can have."""
    return -(-k // 32) * 16, _scale_bytes(fmt, rows, k)


def mx4_layout(rows: int, k: int, fmt: str = "mxfp4"):
    """(bytes of a row of codes, bytes of all scales) of a rows x k matrix."""
    width, scales = ctypes.c_int64(), ctypes.c_int64()
    _ddg._check("dd_mx4_layout", _ddg.load().dd_mx4_layout(_lookup(MX4_FORMATS, fmt, "fmt"), rows, k,
                                                          ctypes.byref(width), ctypes.byref(scales)))
    return width.value, scales.value


def mx4_quantize(x, fmt: str = "mxfp4", cols: bool = False, out: MX4 | None = None, stream=None) -> MX4:
    """The rows of x (float32, bfloat16 or float16), or with cols its columns,
    in 4-bit form.  A K x N right-hand side is quantised with cols=True."""
    f = _lookup(MX4_FORMATS, fmt, "fmt")
    rows, k, ld = _matrix(x, "x")
    t = _type(x.dtype, "x")
    if cols:
        rows, k = k, rows
    if out is None:
        width, scale_bytes = _sizes(f, rows, k)
        codes, scales = _empty((rows, width), dtype=_uint8, device=x.device), _empty(scale_bytes, dtype=_uint8, device=x.device)
        exponents = _empty(rows, dtype=_int32, device=x.device) if f else None
        out = MX4(codes, scales, exponents, rows, k, fmt)
        if stream is not None:
            for part in (codes, scales) + ((exponents,) if f else ()):
                part.record_stream(stream)
        args = codes.data_ptr(), width, scales.data_ptr(), exponents.data_ptr() if f else 0
    else:
        if out.shape != (rows, k) or out.fmt != fmt:
            raise ValueError(f"out must be a {rows} x {k} {fmt} matrix")
        args = out._args("out")[2:]
        _same_device(x, out.codes)
    _call("dd_mx4_quantize", f, t, int(cols), rows, k, x.data_ptr(), ld, *args, _stream(stream, x))
    return out


def mx4_dequantize(q: MX4, dtype=None, out=None, stream=None):
    """The values q stands for, as a rows x k tensor (bfloat16 by default, which holds them exactly)."""
    dtype = dtype or (out.dtype if out is not None else _torch().bfloat16)
    t = _type(dtype, "dtype")
    args = q._args("q")
    out, ld = _like(out, (q.rows, q.k), dtype, q.codes, "out", stream)
    _call("dd_mx4_dequantize", args[1], t, q.rows, q.k, *args[2:], out.data_ptr(), ld, _stream(stream, out))
    return out


def mx4_tile_scales(scales, fmt: str = "mxfp4"):
    """Scale bytes (rows, blocks) in the tiled order of ddgemm.h, padded with
    zeros: for matrices quantised elsewhere, once when they are loaded."""
    torch = _torch()
    per_k = 2 * (4 if _lookup(MX4_FORMATS, fmt, "fmt") == 0 else 8)  # blocks in 256 of k
    rows, blocks = scales.shape
    s = torch.nn.functional.pad(scales, (0, -blocks % per_k, 0, -rows % 128))
    return s.view(s.shape[0] // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def mx4_gemm(a: MX4, b: MX4, dtype=None, out=None, alpha: float = 1.0, stream=None):
    """alpha a b^T for 4-bit matrices a (M x K) and b (N x K) of one format, as
    an M x N tensor (bfloat16 by default)."""
    if a.fmt != b.fmt or a.k != b.k:
        raise ValueError("a and b must share format and k")
    dtype = dtype or (out.dtype if out is not None else _torch().bfloat16)
    t = _type(dtype, "dtype")
    device, fmt, *left = a._args("a")
    other, _, *right = b._args("b")
    if device != other:
        raise ValueError("a and b must be on the same device")
    out, ld = _like(out, (a.rows, b.rows), dtype, a.codes, "out", stream)
    _call("dd_mx4_gemm", fmt, a.rows, b.rows, a.k, *left, *right, alpha, t, out.data_ptr(), ld, _stream(stream, out))
    return out


# ---- the gated block ----

def _ff_shapes(x, Wg, Wu, Wd):
    """(type, T, D, F, the operands' pointers and leading dimensions in turn)."""
    T, D, ldx = _matrix(x, "x")
    dtype = x.dtype
    code = _type(dtype, "x", sixteen=True)
    F, dg, ldg = _matrix(Wg, "Wg", dtype)
    fu, du, ldu = _matrix(Wu, "Wu", dtype)
    dd, fd, ldd = _matrix(Wd, "Wd", dtype)
    if (dg, fu, du, dd, fd) != (D, F, D, D, F):
        raise ValueError("Wg and Wu must be F x D and Wd D x F for x of T x D")
    _same_device(x, Wg, Wu, Wd)
    return code, T, D, F, (x.data_ptr(), ldx, Wg.data_ptr(), ldg, Wu.data_ptr(), ldu, Wd.data_ptr(), ldd)


def ff_gated_saved_size(T: int, F: int, dtype) -> int:
    """Bytes that ff_gated(save=True) keeps for the backward pass."""
    return _saved_size(T, F, _type(dtype, "dtype", sixteen=True))


@functools.lru_cache(maxsize=64)
def _saved_size(T, F, code):
    n = ctypes.c_size_t()
    _ddg._check("dd_ff_gated_saved_size", _ddg.load().dd_ff_gated_saved_size(code, T, F, ctypes.byref(n)))
    return n.value


def ff_gated(x, Wg, Wu, Wd, act: str = "silu", save: bool = False, out=None, stream=None):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T in bfloat16 or float16 (x: T x D, Wg and
    Wu: F x D, Wd: D x F); with save=True (y, saved) for ff_gated_backward."""
    code, T, D, F, operands = _ff_shapes(x, Wg, Wu, Wd)
    a = _lookup(ACTIVATIONS, act, "act")
    y, ldy = _like(out, (T, D), x.dtype, x, "out", stream)
    saved, n = None, 0
    if save:
        n = _saved_size(T, F, code)
        saved = _empty(n, dtype=_uint8, device=x.device)
        if stream is not None:
            saved.record_stream(stream)
    _call("dd_ff_gated", code, a, T, D, F, *operands, y.data_ptr(), ldy, saved.data_ptr() if n else 0, n,
          _stream(stream, x))
    return (y, saved) if save else y


def ff_gated_backward(dy, x, Wg, Wu, Wd, saved, dx=None, dWg=None, dWu=None, dWd=None, need=(True,) * 4, stream=None):
    """(dx, dWg, dWu, dWd) from dy and what ff_gated(save=True) kept; `need` says
    which of them are wanted (None in the place of the others).  Tensors that
    are given are overwritten."""
    code, T, D, F, operands = _ff_shapes(x, Wg, Wu, Wd)
    rows, cols, lddy = _matrix(dy, "dy", x.dtype)
    if (rows, cols) != (T, D):
        raise ValueError("dy must be T x D")
    if not isinstance(saved, _Tensor) or saved.dtype != _uint8 or not saved.is_cuda or not saved.is_contiguous():
        raise TypeError("saved must be the uint8 CUDA tensor that ff_gated returned")
    n = saved.numel()
    if n != _saved_size(T, F, code):
        raise ValueError("saved is of another T, F or type")
    _same_device(x, dy, saved)
    outs, args = [], []
    for name, o, shape, want in zip(("dx", "dWg", "dWu", "dWd"), (dx, dWg, dWu, dWd), ((T, D), (F, D), (F, D), (D, F)), need):
        o, ld = _like(o, shape, x.dtype, x, name, stream) if want else (None, shape[1] or 1)
        outs.append(o)
        args += (o.data_ptr() if want else 0, ld)
    _call("dd_ff_gated_backward", code, T, D, F, dy.data_ptr(), lddy, *operands, saved.data_ptr() if n else 0, n, *args,
          _stream(stream, x))
    return tuple(outs)


def mx4_ff_weights(Wg, Wu, Wd, fmt: str = "mxfp4", stream=None):
    """(w_in, w_out), the weights of mx4_ff_gated from those of ff_gated, once
    when a model is loaded: Wg and Wu in one matrix, 32 rows of each in turn
    (the last groups filled up with zeros), quantised along D, and Wd
    quantised along F."""
    torch = _torch()
    F, D = Wg.shape
    if tuple(Wu.shape) != (F, D) or tuple(Wd.shape) != (D, F):
        raise ValueError("Wg and Wu must be F x D and Wd D x F")
    if stream is not None:  # made in the stream's share of memory, kept while the current one uses them
        current = torch.cuda.current_stream(Wg.device)
        with torch.cuda.stream(stream):
            made = mx4_ff_weights(Wg, Wu, Wd, fmt)
        for part in (t for q in made for t in (q.codes, q.scales, q.exponents) if t is not None):
            part.record_stream(current)
        return made
    pair = [torch.nn.functional.pad(w, (0, 0, 0, -F % 32)).reshape(-1, 32, D) for w in (Wg, Wu)]
    both = torch.stack(pair, 1).view(-1, D)
    return mx4_quantize(both, fmt), mx4_quantize(Wd, fmt)


def mx4_ff_gated(x, w_in: MX4, w_out: MX4, act: str = "silu", out=None, stream=None):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T with 4-bit operands: the weights as
    mx4_ff_weights lays them out, x and the hidden values quantised in the
    call.  x and y: float32, bfloat16 or float16, T x D."""
    T, D, ldx = _matrix(x, "x")
    t = _type(x.dtype, "x")
    a = _lookup(ACTIVATIONS, act, "act")
    F = w_out.k
    if w_in.fmt != w_out.fmt or w_in.k != D or w_out.rows != D or w_in.rows != 2 * (-(-F // 32) * 32):
        raise ValueError("w_in must be 2 * (F rounded up to 32) x D and w_out D x F, of one format")
    device, fmt, *first = w_in._args("w_in")
    other, _, *second = w_out._args("w_out")
    if not device == other == x.get_device():
        raise ValueError("x and the weights must be on the same device")
    y, ldy = _like(out, (T, D), x.dtype, x, "out", stream)
    _call("dd_mx4_ff_gated", fmt, t, a, T, D, F, x.data_ptr(), ldx, *first, *second, y.data_ptr(), ldy,
          _stream(stream, x))
    return y
